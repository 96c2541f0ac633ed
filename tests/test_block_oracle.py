"""The float64 oracle of the operators around the linears (oracle/block.py):
its gradients against central differences of its forward, its 8-bit code
tables against the format's definition, and the host-side tables of the
library (rotation frequencies, AdamW plan) against it.  No GPU."""
import ctypes
import math

import numpy as np
import pytest

from bit_quantized_amd import ops
from oracle import block as OB

H = 1e-6            # central differences: truncation H^2 ~ 1e-12, cancellation 2^-52 / H ~ 2e-10
TOL = 1e-7          # relative to the gradient's scale


def diff(f, x, i):
    a, b = x.copy(), x.copy()
    a.flat[i] += H
    b.flat[i] -= H
    return (f(a) - f(b)) / (2 * H)


def check(f, x, g, rng, n=12):
    scale = np.abs(g).max() + 1e-3
    for i in rng.choice(x.size, size=min(n, x.size), replace=False):
        assert abs(diff(f, x, i) - g.flat[i]) <= TOL * scale * 10, (i, diff(f, x, i), g.flat[i])


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
def test_norm_gradients_against_differences(norm, post):
    rng = np.random.default_rng(1)
    M, C, B = 7, 16, 3
    which = np.array([0, 0, 0, 2, 2, 2, 2])
    x, y = rng.normal(size=(M, C)), rng.normal(size=(M, C))
    gate, scale, shift = (rng.normal(size=(B, C)) for _ in range(3))
    w, pw = rng.normal(size=C), rng.normal(size=C)
    dh, dr = rng.normal(size=(M, C)), rng.normal(size=(M, C))

    def loss(x=x, y=y, gate=gate, scale=scale, shift=shift, w=w, pw=pw):
        r = OB.gated_residual(x, y, which, gate, pw, post, 1e-6, 0.7)
        return (OB.modulated_norm(r, which, scale, shift, w, norm, 1e-6) * dh).sum() + (r * dr).sum()

    r = OB.gated_residual(x, y, which, gate, pw, post, 1e-6, 0.7)
    g = OB.norm_backward(dh, dr, r, y, which, B, gate, scale, w, pw, norm, post, 1e-6, 0.7)
    for name, arg, val in (("dx", "x", x), ("dy", "y", y), ("dgate", "gate", gate), ("dscale", "scale", scale),
                           ("dshift", "shift", shift), ("dweight", "w", w), ("dpost_weight", "pw", pw)):
        check(lambda t: loss(**{arg: t}), val, g[name], rng)
    assert np.all(g["dgate"][1] == 0) and np.all(g["dscale"][1] == 0)      # the sample without rows


@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("normed", [False, True])
def test_rope_gradient_against_differences(layout, normed):
    rng = np.random.default_rng(2)
    M, Hh, D = 5, 2, 24
    angle = OB.rope_angles(rng.integers(-9, 99, (M, 2)), [12, 4], 100.0, "axis")
    x, d = rng.normal(size=(M, Hh, D)), rng.normal(size=(M, Hh, D))
    w = rng.normal(size=D) if normed else None
    loss = lambda x=x, w=w: (OB.rope_forward(x, angle, layout, w, 1e-6) * d).sum()
    dx, dw = OB.rope_backward(d, x, angle, layout, w, 1e-6)
    check(lambda t: loss(x=t), x, dx, rng)
    if normed:
        check(lambda t: loss(w=t), w, dw, rng)


@pytest.mark.parametrize("mask, cap", [("full", 0.0), ("causal", 0.0), ("prefix", 3.0), ("full", 2.0)])
def test_attention_gradient_against_differences(mask, cap):
    rng = np.random.default_rng(3)
    n, D = 6, 8
    q, k, v, do = (rng.normal(size=(n, D)) for _ in range(4))
    see = OB.visible(n, mask, 3)
    loss = lambda q=q, k=k, v=v: (OB.attention_head(q, k, v, see, 0.4, cap)[0] * do).sum()
    o, lse, p, slope = OB.attention_head(q, k, v, see, 0.4, cap)
    dq, dk, dv, _ = OB.attention_head_grad(q, k, v, do, o, p, slope, 0.4)
    for arg, val, g in (("q", q, dq), ("k", k, dk), ("v", v, dv)):
        check(lambda t: loss(**{arg: t}), val, g, rng)
    assert np.allclose(p.sum(1), 1) and np.all(p[~see] == 0)


def test_visible_keys():
    assert OB.visible(3, "causal", 9).tolist() == [[True, False, False], [True, True, False], [True, True, True]]
    assert OB.visible(3, "prefix", 2).tolist() == [[True, True, False], [True, True, False], [True, True, True]]
    assert OB.visible(2, "full", 0).all()


def test_adamw_against_its_definition():
    """One step from zero states moves every element by lr (1 + eps' effects) against its gradient's sign."""
    p, m, v = OB.adamw(np.array([1.0, -2.0]), np.array([3.0, -1e-3]), np.zeros(2), np.zeros(2), 1, 0.1, 0.9, 0.999,
                       1e-12, 0.0)
    np.testing.assert_allclose(p, [0.9, -1.9], rtol=1e-9)
    np.testing.assert_allclose(m, [0.3, -1e-4])
    np.testing.assert_allclose(v, [9e-3, 1e-9])


@pytest.mark.parametrize("signed", [True, False])
def test_code_values(signed):
    v = OB.code_values(signed)
    half = v[:128] if signed else v
    assert half[0] == 0 and half[-1] == 1 and np.all(np.diff(half) > 0)
    assert len(v) == 256 and (not signed or np.array_equal(v[128:], -v[:128]))
    # 4 fraction bits: neighbouring codes are at most 1/16 apart above the lowest exponent
    assert np.all(np.diff(half)[16:] / half[16:-1] <= 1 / 16 + 1e-12)
    # values that codes stand for come back as those codes, whatever the random bits
    for bits in (0, 2 ** 19 - 1):
        c = OB.code_round(v * 3.0, 3.0, np.full(256, bits), signed)
        assert np.array_equal(OB.code_values(signed)[c], v)


def test_random_bits_are_even():
    h = np.array([OB.mixed_bits(i, 7, 3) for i in range(20000)]) / 2.0 ** 32
    # mean and variance of 20000 uniform values: 5 deviations of either
    assert abs(h.mean() - 0.5) < 5 * math.sqrt(1 / 12 / 20000)
    assert abs(h.var() - 1 / 12) < 5 * math.sqrt(1 / 180 / 20000)
    assert abs(np.corrcoef(h[:-1], h[1:])[0, 1]) < 5 / math.sqrt(20000)


# ------------------------------------------------------------ the library's host side
@pytest.mark.parametrize("ladder", ["axis", "shared"])
def test_rope_table(ladder):
    dims = [16, 56, 40]
    rp = ops.fourtune_rope_init(128, dims, 10000.0, ops.FT_ROPE_HALVES,
                                {"axis": ops.FT_ROPE_AXIS, "shared": ops.FT_ROPE_SHARED}[ladder])
    assert rp.n_pairs == 56 and list(rp.axis[:56]) == [0] * 8 + [1] * 28 + [2] * 20
    want = OB.rope_angles(np.ones((1, 3)), dims, 10000.0, ladder)[0] / (2 * math.pi)
    got = np.array(rp.turn_hi[:56], dtype=np.float64) + np.array(rp.turn_lo[:56], dtype=np.float64)
    np.testing.assert_allclose(got, want, rtol=2.0 ** -46)


def test_adamw_plan_places():
    n = [5, 0, 128, 129, 4096]
    t = (ops.FtAdamwTensor * 5)(*[ops.FtAdamwTensor(0x1000 * (i + 1), 0x100000 * (i + 1), None, k) for i, k in enumerate(n)])
    size, arena = ops.fourtune_adamw_plan_bytes(t, 5)
    assert arena == 128 + 0 + 128 + 256 + 4096
    host = (ctypes.c_uint8 * size)()
    d = ops.fourtune_adamw_plan(t, 5, ops.FT_F32, ops.FT_BF16, ops.FT_STATE_F32, ctypes.addressof(host), size)
    assert (d.n_tensors, d.arena, d.n_chunks, d.has_master) == (5, arena, 1 + 0 + 1 + 1 + 2, 0)
