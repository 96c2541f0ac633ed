"""GPU: the operators around the linears against the float64 oracle
(oracle/block.py) on the same bf16 or fp32 inputs, elementwise.

Bounds.  Every output is one rounding to its type (half a step of the type at
the exact value) of a value computed in fp32 from the inputs.  DEPTH * 2^-24
times the sum of the magnitudes of the terms bounds the fp32 part: DEPTH =
256 covers the longest chain of fp32 additions any term goes through here (at
most 64 rows or 32 partial sums one after the other, trees of 6 and 4 levels,
a dozen operations per term).  The rotation adds 2^-18 for the hardware's
sine and cosine (2^-19 each).  In attention the probabilities and their
gradients enter a matrix product rounded to bf16 (8 bits, so half a step is
up to 2^-8 of the value) and a query of more than 1024 keys takes delta from
the output rounded to bf16, 2^-8 of each product in do . o.
"""
import numpy as np
import pytest
import torch

from bit_quantized_amd import block, ops
from oracle import block as OB

from _gpu import DEV, require_gpu, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEPTH = 256


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def f64(t):
    return t.detach().double().cpu().numpy()


def draw(rng, *shape, std=1.0, dtype=BF):
    return torch.from_numpy(rng.normal(size=shape) * std).to(dtype).to(DEV)


def close(got, exact, mag, what, extra=0.0):
    """got within half a step of its type, DEPTH 2^-24 mag and `extra` of exact."""
    mant = 8 if got.dtype == BF else 24
    g, exact = f64(got), np.asarray(exact)
    assert g.shape == exact.shape, (what, g.shape, exact.shape)
    assert np.isfinite(g).all(), (what, "not finite")
    bound = OB.half_step(exact, mant) * (1 + 1e-6) + DEPTH * 2.0 ** -24 * np.asarray(mag) + extra + 1e-37
    far = np.abs(g - exact) > bound
    if far.any():
        raise AssertionError((what, int(far.sum()), np.argwhere(far)[:4].tolist(), g[far][:4], exact[far][:4],
                              np.broadcast_to(bound, g.shape)[far][:4]))


# ------------------------------------------------------------------ norm
def _norm_case(rows, C, norm, post, stream, factors, alpha, seed, uniform=False):
    rng = np.random.default_rng(seed)
    M, B = sum(rows), len(rows)
    x = draw(rng, M, C, dtype=stream) + 0.25
    y = None if post is None else draw(rng, M, C, std=0.7)
    mod = draw(rng, B, 3 * C, std=0.5)
    f = dict(gate=mod[:, :C], scale=mod[:, C:2 * C], shift=mod[:, 2 * C:])
    f = {k: v for k, v in f.items() if k in factors}
    if post is None:
        f.pop("gate", None)
    w = draw(rng, C) if "weight" in factors else None
    pw = draw(rng, C) if "post_weight" in factors and post is not None else None
    seg = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=DEV)
    op = block.GatedNorm(norm=norm, post_norm=post or "none", weight=w, post_weight=pw, eps=1e-5, alpha=alpha)
    which = OB.samples_of(np.concatenate([[0], np.cumsum(rows)]), M)
    full = lambda k, none: f64(f[k]) if k in f else np.full((B, C), none)
    o = dict(gate=full("gate", 1.0), scale=full("scale", 0.0), shift=full("shift", 0.0),
             w=np.ones(C) if w is None else f64(w), pw=np.ones(C) if pw is None else f64(pw))
    return rng, op, x, y, f, (None if uniform else seg), which, B, o


ALL = ("gate", "scale", "shift", "weight", "post_weight")
NORM_CASES = [
    # rows of the samples, channels, norm, post (None: no y), stream, factors, alpha
    ((1,), 8, "layer", None, BF, ("scale", "shift"), 1.0),
    ((3,), 1160, "rms", "rms", F32, ALL, 1.0),
    ((0, 5, 0, 0, 12, 1), 136, "layer", "layer", BF, ALL, 0.5),
    ((700, 1, 349), 512, "layer", "none", BF, ("gate", "scale", "shift"), 1.0),      # two rows a workgroup
    ((1024, 1), 520, "rms", "layer", F32, ("gate", "weight"), -2.0),
    ((9,), 4104, "layer", "rms", BF, ALL, 1.0),
    ((1030,), 4104, "rms", "none", F32, (), 1.0),
    ((40, 2), 8200, "layer", "rms", F32, ALL, 1.0),
    ((11,), 16384, "rms", "layer", BF, ALL, 1.0),
    ((64,) * 5, 72, "layer", None, F32, ("scale",), 1.0),
]


@pytest.mark.parametrize("case", NORM_CASES, ids=lambda c: "%dx%d-%s-%s" % (sum(c[0]), c[1], c[2], c[3]))
@pytest.mark.parametrize("grad_f32", [False, True])
def test_norm(case, grad_f32):
    rows, C, norm, post, stream, factors, alpha = case
    say("norm", case, grad_f32)
    rng, op, x, y, f, seg, which, B, o = _norm_case(*case, seed=C + len(rows))
    M = sum(rows)
    r, h, stats = op.forward(x, y=y, segments=seg, **f)
    X = f64(x)
    if y is None:
        assert r is x
    else:
        n, _, _ = OB.norm_rows(f64(y), post, 1e-5)
        exact = OB.gated_residual(X, f64(y), which, o["gate"], o["pw"], post, 1e-5, alpha)
        close(r, exact, np.abs(X) + np.abs(alpha * o["gate"][which] * o["pw"]) * (np.abs(n) + 1), "r")
    R = f64(r)
    n, mean, rstd = OB.norm_rows(R, norm, 1e-5)
    exact = OB.modulated_norm(R, which, o["scale"], o["shift"], o["w"], norm, 1e-5)
    close(h, exact, np.abs(1 + o["scale"][which]) * np.abs(o["w"]) * (np.abs(n) + np.abs(mean) * rstd + 1)
          + np.abs(o["shift"][which]), "h")
    close(stats[:, :2], np.concatenate([mean, rstd], 1), np.abs(R).mean(1, keepdims=True) + rstd, "stats")

    dh, dr = draw(rng, M, C, std=1e-2), draw(rng, M, C, std=1e-2, dtype=stream)
    g = op.backward(dh, dr, r, y, stats, segments=seg, grad_f32=grad_f32, **f)
    e = OB.norm_backward(f64(dh), f64(dr), R, None if y is None else f64(y), which, B, o["gate"], o["scale"], o["w"],
                         o["pw"], norm, post or "none", 1e-5, alpha)
    want = {"dx"} | ({"dy"} if y is not None else set()) | {"d" + k for k in f}
    want |= {"dweight"} & ({"dweight"} if op.weight is not None else set())
    want |= {"dpost_weight"} & ({"dpost_weight"} if op.post_weight is not None else set())
    assert {k for k, v in g.items() if v is not None} == want
    # (n itself carries the fp32 error of mean and rstd into every product with it)
    for k in sorted(want):
        assert g[k].dtype == (stream if k == "dx" else BF if k == "dy" else F32 if grad_f32 else BF)
        off = (np.abs(mean) * rstd + 1).max()
        close(g[k], e[k], e["|" + k] * off, k)
    # the same bits again
    r2, h2, _ = op.forward(x, y=y, segments=seg, **f)
    g2 = op.backward(dh, dr, r2, y, stats, segments=seg, grad_f32=grad_f32, **f)
    assert torch.equal(h, h2) and all(torch.equal(g[k], g2[k]) for k in want)


def test_norm_gradient_against_differences():
    """The kernels' gradient along a random direction against central differences of the oracle's
    forward (fp32 stream; the norm's own rounding of r is 2^-24)."""
    rng, op, x, y, f, seg, which, B, o = _norm_case((5, 3), 64, "layer", "rms", F32, ALL, 1.0, seed=5)
    r, h, stats = op.forward(x, y=y, segments=seg, **f)
    dh, dr = draw(rng, 8, 64), draw(rng, 8, 64, dtype=F32)
    g = op.backward(dh, dr, r, y, stats, segments=seg, grad_f32=True, **f)

    def loss(X, Y, gate):
        rr = OB.gated_residual(X, Y, which, gate, o["pw"], "rms", 1e-5, 1.0)
        return (OB.modulated_norm(rr, which, o["scale"], o["shift"], o["w"], "layer", 1e-5) * f64(dh)).sum() + (rr * f64(dr)).sum()

    X, Y = f64(x), f64(y)
    for k, name in enumerate(("dx", "dy", "dgate")):
        d = rng.normal(size=f64(g[name]).shape)
        step = lambda t: [(X, Y, o["gate"])[i] + (t * d if i == k else 0) for i in range(3)]
        slope = (loss(*step(1e-5)) - loss(*step(-1e-5))) / 2e-5
        # dy is bf16: 2^-8 of each term; differences: 1e-10 relative third order and 1e-11 / 1e-5 cancellation
        bound = (2.0 ** -8 if name == "dy" else 2.0 ** -15) * np.abs(f64(g[name]) * d).sum() + 1e-5 * abs(slope) + 1e-5
        assert abs((f64(g[name]) * d).sum() - slope) <= bound, name


def test_norm_special_rows():
    """Rows without variance, one modulation for all, uniform samples, a residual alone, results in
    place, an empty batch."""
    C, M = 256, 6
    rng = np.random.default_rng(9)
    op = block.GatedNorm(norm="layer", eps=1e-6)
    x = torch.full((M, C), 3.0, dtype=BF, device=DEV)
    mod = draw(rng, 3, C)
    r, h, stats = op.forward(x, scale=mod, shift=mod)              # rows constant: n = 0, h = shift
    assert torch.equal(h, mod.repeat_interleave(2, 0))
    y = draw(rng, M, C)
    r, h, _ = op.forward(x, y=y, gate=mod[:1], need_h=False)
    assert h is None
    close(r, f64(x) + f64(mod[:1]) * f64(y), np.abs(f64(y) * f64(mod[:1])) + 3, "r")
    g = op.backward(None, r, r, y, None, gate=mod[:1])             # dr alone
    assert torch.equal(g["dx"], r) and g["dscale"] is None
    # in place: r over x, dx over dr
    x1, x2 = draw(rng, M, C), None
    x2 = x1.clone()
    want = op.forward(x1, y=y, scale=mod, shift=mod, gate=mod)
    st = torch.empty((M, 4), dtype=F32, device=DEV)
    h = torch.empty_like(x1)
    ops.fourtune_norm_fwd(op.desc(x2, mod, mod, mod), x2, y, x2, h, st)
    assert torch.equal(x2, want[0]) and torch.equal(h, want[1])
    dh, dr = draw(rng, M, C), draw(rng, M, C)
    ref = op.backward(dh, dr, want[0], y, st, mod, mod, mod)
    dy = torch.empty_like(y)
    ops.fourtune_norm_bwd(op.desc(x2, mod, mod, mod), dh, dr, x2, y, st, dr, dy, None, None, None, C, None, None, 0, None, 0)
    assert torch.equal(dr, ref["dx"]) and torch.equal(dy, ref["dy"])
    # no rows: outputs of no rows, gradients of zero
    e = x1[:0]
    seg = torch.zeros(3, dtype=torch.int32, device=DEV)
    r, h, st = op.forward(e, y=e, gate=mod[:2], scale=mod[:2], shift=mod[:2], segments=seg)
    g = op.backward(e, e, r, e, st, gate=mod[:2], scale=mod[:2], shift=mod[:2], segments=seg)
    assert h.shape == (0, C) and all(float(g[k].float().abs().sum()) == 0 for k in ("dgate", "dscale", "dshift"))


# ------------------------------------------------------------------ rope
ROPE_CASES = [
    # rows, q heads, k heads, D, axis dims, layout, ladder, normed, position range
    (1, 1, 1, 8, (8,), "pairs", "axis", False, (0, 10)),
    (77, 12, 4, 64, (64,), "halves", "axis", False, (0, 77)),
    (5, 3, 1, 72, (24, 24, 24), "pairs", "shared", True, (0, 5000)),
    (33, 2, 0, 128, (16, 56, 56), "pairs", "axis", True, (-300, 300)),
    (130, 5, 5, 96, (32, 32), "halves", "shared", True, (0, 16384)),      # a third of the head passes through
    (257, 4, 2, 256, (2, 4, 6, 244), "pairs", "axis", True, (0, 1000)),
    (2050, 2, 2, 128, (128,), "halves", "axis", True, (0, 1 << 20)),
    (9, 1, 40, 40, (10, 6), "pairs", "axis", False, (0, 1 << 24)),
]


@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: "%dx%d+%dx%d-%s" % (c[0], c[1], c[2], c[3], c[5]))
def test_rope(case):
    M, hq, hk, D, dims, layout, ladder, normed, (lo, hi) = case
    say("rope", case)
    rng = np.random.default_rng(M + D)
    wq, wk = (draw(rng, D) if normed else None for _ in range(2))
    op = block.AxialRotary(D, dims, theta=10000.0, layout=layout, ladder=ladder, q_weight=wq, k_weight=wk, eps=1e-6)
    qkv = draw(rng, M, (hq + 2 * max(hk, 1)) * D)
    q = qkv[:, :hq * D].unflatten(1, (hq, D))
    k = qkv[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D)) if hk else torch.empty((M, 0, D), dtype=BF, device=DEV)
    pos = torch.from_numpy(rng.integers(lo, hi, (M, len(dims)))).int().to(DEV)
    angle = OB.rope_angles(pos.cpu().numpy(), dims, 10000.0, ladder)
    q2, k2 = op.forward(q, k, pos)
    dq, dk = draw(rng, M, hq, D), draw(rng, M, hk, D)
    g = op.backward(dq, dk, q, k, pos, grad_f32=True)
    for n, x, y, w, d in (("q", q, q2, wq, dq), ("k", k, k2, wk, dk)):
        if x.shape[1] == 0:
            assert g["dw" + n] is None
            continue
        W = None if w is None else f64(w)
        t = np.abs(f64(x)) if W is None else np.abs(W * f64(x)) / np.sqrt((f64(x) ** 2).mean(2, keepdims=True) + 1e-6)
        mag = _pair_mag(t, len(angle[0]), layout)
        close(y, OB.rope_forward(f64(x), angle, layout, W, 1e-6), mag, n, extra=2.0 ** -18 * mag)
        ex, ew = OB.rope_backward(f64(d), f64(x), angle, layout, W, 1e-6)
        u = _pair_mag(np.abs(f64(d)), len(angle[0]), layout)
        if W is None:
            close(g["d" + n], ex, u, "d" + n, extra=2.0 ** -18 * u)
        else:
            rstd = 1 / np.sqrt((f64(x) ** 2).mean(2, keepdims=True) + 1e-6)
            nn = np.abs(f64(x)) * rstd
            a = u * np.abs(W)
            m = rstd * (a + nn * (a * nn).mean(2, keepdims=True))
            close(g["d" + n], ex, m, "d" + n, extra=2.0 ** -18 * m)
            s = (u * nn).sum((0, 1))
            close(g["dw" + n], ew, s, "dw" + n, extra=2.0 ** -18 * s)
    # in place, and the gradient in place, give the same bits
    buf = qkv.clone()
    qb = buf[:, :hq * D].unflatten(1, (hq, D))
    kb = buf[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D)) if hk else k
    op.forward(qb, kb, pos, qb, kb)
    assert torch.equal(qb, q2) and torch.equal(kb, k2) and torch.equal(buf[:, (hq + hk) * D:], qkv[:, (hq + hk) * D:])
    op.backward(dq, dk, q, k, pos, dq, dk, need_weights=False)
    assert torch.equal(dq, g["dq"]) and torch.equal(dk, g["dk"])


def _pair_mag(t, pairs, layout):
    """|a| + |b| of each value's pair; a value past the pairs itself."""
    out = t.copy()
    for j in range(pairs):
        a, b = (2 * j, 2 * j + 1) if layout == "pairs" else (j, j + pairs)
        out[:, :, a] = out[:, :, b] = t[:, :, a] + t[:, :, b]
    return out


def test_rope_without_rows():
    w = torch.ones(64, dtype=BF, device=DEV)
    op = block.AxialRotary(64, [64], q_weight=w, k_weight=w)
    e, pos = torch.empty((0, 2, 64), dtype=BF, device=DEV), torch.empty((0, 1), dtype=torch.int32, device=DEV)
    q, k = op.forward(e, e, pos)
    g = op.backward(e, e, e, e, pos)
    assert q.shape == (0, 2, 64) and float(g["dwq"].abs().sum()) == 0 and float(g["dwk"].abs().sum()) == 0


# ------------------------------------------------------------------ attention
ATTN_CASES = [
    # documents, rows before and after them, q heads, k heads, D, mask, cap
    ((1,), (0, 0), 1, 1, 64, "full", 0.0),
    ((1, 1, 0, 2, 3), (2, 1), 4, 2, 128, "causal", 0.0),
    ((31, 32, 33, 0, 63, 64, 65), (0, 5), 2, 1, 64, "full", 0.0),
    ((127, 128, 129), (3, 0), 2, 2, 128, "prefix", 0.0),
    ((255, 257, 1), (0, 0), 3, 1, 128, "full", 30.0),
    ((300, 17), (1, 1), 4, 4, 64, "causal", 2.0),
    ((640, 0, 77), (0, 19), 6, 2, 64, "prefix", 50.0),
    ((1300,), (0, 0), 1, 1, 64, "causal", 0.0),                        # more than 1024 keys
    ((1100,), (0, 0), 2, 1, 128, "full", 0.0),
    (tuple(range(1, 75)), (0, 2), 1, 1, 64, "causal", 0.0),            # more than 64 documents
]


def _heads64(t):
    return f64(t).transpose(1, 0, 2)


def _attn_check(q, k, v, do, o, lse, dq, dk, dv, starts, prefix, mask, cap, heads=None):
    M, Hq, D = q.shape
    Hk = k.shape[1]
    scale = D ** -0.5
    Q, K, V, G = _heads64(q), _heads64(k), _heads64(v), _heads64(do)
    zero = lambda h: np.zeros((h, M, D))
    eo, edq, edk, edv = zero(Hq), zero(Hq), zero(Hk), zero(Hk)
    bo, bdq, bdk, bdv = zero(Hq), zero(Hq), zero(Hk), zero(Hk)
    els, bls = np.full((Hq, M), -np.inf), np.zeros((Hq, M))
    e = 2.0 ** -8 * 1.01
    for d, (a, b) in enumerate(zip(starts, starts[1:])):
        if a == b:
            continue
        see = OB.visible(b - a, mask, prefix[d])
        for h in range(Hq):
            g = h // (Hq // Hk)
            qq, kk, vv, gg = Q[h, a:b], K[g, a:b], V[g, a:b], G[h, a:b]
            oo, ll, p, slope = OB.attention_head(qq, kk, vv, see, scale, cap)
            x, y, z, ds = OB.attention_head_grad(qq, kk, vv, gg, oo, p, slope, scale)
            eo[h, a:b], els[h, a:b], edq[h, a:b] = oo, ll, x
            edk[g, a:b] += y
            edv[g, a:b] += z
            # fp32 scores: off by at most this, and p by that relative amount
            so = 64 * 2.0 ** -24 * scale * (np.abs(qq) @ np.abs(kk).T).max(1, keepdims=True) + (5e-7 * cap if cap else 0) + 2.0 ** -20
            pr = e + 2 * so
            bo[h, a:b] = (pr * p) @ np.abs(vv)
            bls[h, a:b] = so[:, 0] + 2.0 ** -22 * np.abs(ll)
            dp = np.abs(gg) @ np.abs(vv).T
            w = p * slope * (2 * so * np.abs(gg @ vv.T - (gg * oo).sum(1, keepdims=True)) + DEPTH * 2.0 ** -24 * (dp + np.abs(gg * oo).sum(1, keepdims=True)))
            few = see.sum(1, keepdims=True) <= 960          # a tile of 128 or 256 queries with at most 1024 keys
            w = w + p * slope * np.where(few, 0, 2.0 ** -8 * np.abs(gg * oo).sum(1, keepdims=True))
            w = w + e * np.abs(ds)
            bdq[h, a:b] = scale * w @ np.abs(kk)
            bdk[g, a:b] += scale * w.T @ np.abs(qq)
            bdv[g, a:b] += (pr * p).T @ np.abs(gg)
    T = lambda t: t.transpose(1, 0, 2)
    close(o, T(eo), T(np.abs(eo)), "o", extra=T(bo))
    L = f64(lse)
    assert np.array_equal(np.isneginf(L), np.isneginf(els)), "lse of empty rows"
    fin = np.isfinite(els)
    assert np.all(np.abs(L[fin] - els[fin]) <= bls[fin]), ("lse", np.abs(L[fin] - els[fin]).max())
    close(dq, T(edq), T(np.abs(edq)), "dq", extra=T(bdq))
    close(dk, T(edk), T(np.abs(edk)), "dk", extra=T(bdk))
    close(dv, T(edv), T(np.abs(edv)), "dv", extra=T(bdv))


@pytest.mark.parametrize("case", ATTN_CASES, ids=lambda c: "%ddocs-%d-%dof%d-D%d-%s-%g" % (len(c[0]), sum(c[0]), c[2], c[3], c[4], c[5], c[6]))
def test_attention(case):
    docs, (before, after), Hq, Hk, D, mask, cap = case
    say("attention", case if len(docs) < 20 else (len(docs),) + case[1:])
    rng = np.random.default_rng(sum(docs) + D)
    M = sum(docs) + before + after
    starts = np.concatenate([[0], np.cumsum(docs)]) + before
    qkv = draw(rng, M, (Hq + 2 * Hk) * D, std=1.2)
    q, k, v = block.split_qkv(qkv, Hq, Hk, D)                           # strided parts of one tensor
    do = draw(rng, M, Hq, D)
    # what lies in no document does not count, whatever it is
    for t in (qkv, do):
        t[:before] = float("nan")
        t[M - after:] = float("inf")
    off = torch.tensor(starts, dtype=torch.int32, device=DEV)
    pre = torch.tensor([n // 3 if i % 2 else n + 7 for i, n in enumerate(docs)], dtype=torch.int32, device=DEV)
    op = block.DocAttention(D, mask=mask, softcap=cap)
    o, lse = op.forward(q, k, v, docs=off, prefix=pre)
    dqkv = torch.full_like(qkv, float("nan"))
    dq, dk, dv = op.backward(do, q, k, v, o, lse, off, pre, *block.split_qkv(dqkv, Hq, Hk, D))
    inside = torch.zeros(M, 1, 1, dtype=torch.bool, device=DEV)
    inside[before:M - after] = True
    z = lambda t: torch.where(inside, t, torch.zeros_like(t))
    _attn_check(z(q), z(k), z(v), z(do), o, lse, dq, dk, dv, starts, pre.tolist(), mask, cap)
    assert float(o[:before].float().abs().sum()) == 0 and float(dqkv[M - after:].float().abs().sum()) == 0
    o2, _ = op.forward(q, k, v, docs=off, prefix=pre, need_lse=False)
    g2 = op.backward(do, q, k, v, o, lse, off, pre)
    assert torch.equal(o, o2) and all(torch.equal(a, b) for a, b in zip((dq, dk, dv), g2))      # the same bits


@pytest.mark.parametrize("D", [64, 128])
def test_attention_wide_workgroups(D):
    """Heads enough that the kernels take 256 queries a workgroup: against the oracle on some heads."""
    M, Hq, Hk = 1100, 96, 48
    rng = np.random.default_rng(D)
    q, k, v, do = draw(rng, M, Hq, D), draw(rng, M, Hk, D), draw(rng, M, Hk, D), draw(rng, M, Hq, D)
    starts = [0, 300, 301, 900, 1100]
    off = torch.tensor(starts, dtype=torch.int32, device=DEV)
    op = block.DocAttention(D, mask="causal")
    o, lse = op.forward(q, k, v, docs=off)
    dq, dk, dv = op.backward(do, q, k, v, o, lse, docs=off)
    for g in (0, 31, 47):
        hs = slice(2 * g, 2 * g + 2)
        gs = slice(g, g + 1)
        _attn_check(q[:, hs], k[:, gs], v[:, gs], do[:, hs], o[:, hs], lse[hs], dq[:, hs], dk[:, gs], dv[:, gs], starts,
                    [0] * 4, "causal", 0.0)


@pytest.mark.parametrize("D,mask,cap", [(64, "full", 0.0), (64, "prefix", 20.0), (128, "full", 20.0), (128, "prefix", 0.0)])
def test_attention_wide_workgroups_masks(D, mask, cap):
    """The same with other masks and a cap; documents of one tile and of several, none longer than the last tile."""
    M, H = 600, 96
    rng = np.random.default_rng(D + len(mask))
    q, k, v, do = (draw(rng, M, H, D) for _ in range(4))
    starts, prefix = [0, 1, 65, 257, 257, 600], [1, 64, 70, 0, 150]
    off = torch.tensor(starts, dtype=torch.int32, device=DEV)
    pre = torch.tensor(prefix, dtype=torch.int32, device=DEV) if mask == "prefix" else None
    op = block.DocAttention(D, mask=mask, softcap=cap)
    o, lse = op.forward(q, k, v, docs=off, prefix=pre)
    dq, dk, dv = op.backward(do, q, k, v, o, lse, docs=off, prefix=pre)
    for h in (0, 50, 95):
        s = slice(h, h + 1)
        _attn_check(q[:, s], k[:, s], v[:, s], do[:, s], o[:, s], lse[s], dq[:, s], dk[:, s], dv[:, s], starts,
                    prefix if pre is not None else [0] * 5, mask, cap)


@pytest.mark.parametrize("D,M,Hq,Hk,mask,cap", [
    (64, 40, 4, 2, "causal", 0.0), (128, 100, 2, 1, "prefix", 0.0),            # two groups of one wave
    (64, 700, 2, 1, "prefix", 20.0), (128, 700, 2, 2, "causal", 20.0),         # four groups of one wave
    (64, 260, 20, 10, "full", 0.0), (128, 330, 32, 16, "prefix", 0.0),         # two groups of 64 rows
    (64, 900, 24, 24, "full", 20.0), (128, 700, 20, 20, "causal", 0.0),        # two groups of 128 rows
    (64, 1400, 36, 36, "causal", 0.0), (128, 900, 40, 20, "full", 0.0),        # 128 rows, one group or two
])
def test_attention_by_the_size_of_the_problem(D, M, Hq, Hk, mask, cap):
    """The workgroups' shapes go by the rows times the heads; a document of them ends inside every kind of tile."""
    rng = np.random.default_rng(M + Hq)
    q, k, v, do = draw(rng, M, Hq, D), draw(rng, M, Hk, D), draw(rng, M, Hk, D), draw(rng, M, Hq, D)
    prefix = torch.tensor([M // 3], dtype=torch.int32, device=DEV) if mask == "prefix" else None
    op = block.DocAttention(D, mask=mask, softcap=cap)
    o, lse = op.forward(q, k, v, prefix=prefix)
    dq, dk, dv = op.backward(do, q, k, v, o, lse, prefix=prefix)
    for g in {0, Hk - 1}:
        r = Hq // Hk
        hs, gs = slice(r * g, r * g + r), slice(g, g + 1)
        _attn_check(q[:, hs], k[:, gs], v[:, gs], do[:, hs], o[:, hs], lse[hs], dq[:, hs], dk[:, gs], dv[:, gs], [0, M],
                    [M // 3 if prefix is not None else 0], mask, cap)
    o2, _ = op.forward(q, k, v, prefix=prefix, need_lse=False)
    assert torch.equal(o, o2) and all(torch.equal(a, b) for a, b in zip((dq, dk, dv), op.backward(do, q, k, v, o, lse, prefix=prefix)))


def test_attention_documents_do_not_touch():
    """NaN and Inf in one document leave the others' bits as they are."""
    M, H, D = 400, 2, 64
    rng = np.random.default_rng(4)
    off = torch.tensor([0, 100, 229, 400], dtype=torch.int32, device=DEV)
    op = block.DocAttention(D)
    q, k, v, do = (draw(rng, M, H, D) for _ in range(4))
    res = []
    for poison in (False, True):
        t = [x.clone() for x in (q, k, v, do)]
        if poison:
            for x, bad in zip(t, (float("nan"), float("inf"), float("nan"), -float("inf"))):
                x[100:229] = bad
        o, lse = op.forward(*t[:3], docs=off)
        res.append((o, lse.t(), *op.backward(t[3], *t[:3], o, lse, docs=off)))
    for a, b in zip(*res):
        for s in (slice(0, 100), slice(229, 400)):
            assert torch.equal(a[s], b[s])


def test_attention_gradient_against_differences():
    """The kernels' gradient along random directions against central differences of the oracle's forward."""
    rng = np.random.default_rng(11)
    n, D = 40, 64
    q, k, v, do = (draw(rng, n, 1, D) for _ in range(4))
    op = block.DocAttention(D, mask="causal", softcap=5.0)
    o, lse = op.forward(q, k, v)
    g = op.backward(do, q, k, v, o, lse)
    see = OB.visible(n, "causal", 0)
    base = [f64(t)[:, 0] for t in (q, k, v)]
    for i in range(3):
        d = rng.normal(size=(n, D))
        at = lambda t: [b + (t * d if j == i else 0) for j, b in enumerate(base)]
        loss = lambda t: (OB.attention_head(*at(t), see, D ** -0.5, 5.0)[0] * f64(do)[:, 0]).sum()
        slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
        got = f64(g[i])[:, 0]
        # three bf16 roundings of the gradient's parts, each at most 2^-8 and of either sign: 4 deviations
        assert abs((got * d).sum() - slope) <= 4 * 3 * 2.0 ** -8 * np.linalg.norm(got * d) + 1e-4


def test_attention_offsets_past_32_bits():
    """Rows whose byte offsets pass 2^32: a document at the far end of a long, wide tensor."""
    M, ld, D = 300_000, 9216, 64
    rng = np.random.default_rng(12)
    wide = torch.zeros((M, ld), dtype=BF, device=DEV)
    tail = draw(rng, 150, 3 * D)
    wide[M - 150:, ld - 3 * D:] = tail
    q, k, v = (wide[:, ld - (3 - i) * D:ld - (2 - i) * D or None].unflatten(1, (1, D)) for i in range(3))
    off = torch.tensor([M - 150, M], dtype=torch.int32, device=DEV)
    op = block.DocAttention(D)
    o, lse = op.forward(q, k, v, docs=off)
    sq, sk, sv = (tail[:, i * D:(i + 1) * D].unflatten(1, (1, D)) for i in range(3))
    assert float(o[:M - 150].float().abs().max()) == 0
    grads = op.backward(o, q, k, v, o, lse, docs=off)
    assert all(float(t[:M - 150].float().abs().max()) == 0 for t in grads)
    to = o[M - 150:]
    _attn_check(sq, sk, sv, to, to, lse[:, M - 150:], *(t[M - 150:] for t in grads), [0, 150], [0], "full", 0.0)
    # the rotation and the norm on the same rows
    rot = block.AxialRotary(D, [D])
    pos = torch.arange(M, dtype=torch.int32, device=DEV)[:, None].contiguous()
    a, b = rot.forward(q, k, pos)
    c, d = rot.forward(sq, sk, pos[M - 150:])
    assert torch.equal(a[M - 150:], c) and torch.equal(b[M - 150:], d)
    norm = block.GatedNorm()
    _, h, _ = norm.forward(wide)
    _, h2, _ = norm.forward(wide[M - 150:].contiguous())
    assert torch.equal(h[M - 150:], h2)


def test_more_rows_than_one_grid_axis():
    """Row counts past what one axis of a grid of workgroups counts."""
    norm = block.GatedNorm()
    x = torch.randn(2_200_003, 8, dtype=F32, device=DEV).to(BF)
    _, h, _ = norm.forward(x)
    for a in (0, 2_097_000, 2_198_000):
        _, part, _ = norm.forward(x[a:a + 2003].contiguous())
        assert torch.equal(h[a:a + 2003], part)
    rot = block.AxialRotary(8, [8])
    M = (1 << 24) + 5
    pos = (torch.arange(M, dtype=torch.int32, device=DEV) % 1000)[:, None].contiguous()
    q = x[:, :8].repeat(8, 1)[:M].unflatten(1, (1, 8))
    a, b = rot.forward(q, q, pos)
    for s in (slice(0, 100), slice((1 << 23) - 50, (1 << 23) + 50), slice(M - 100, M)):
        c, d = rot.forward(q[s].contiguous(), q[s].contiguous(), pos[s].contiguous())
        assert torch.equal(a[s], c) and torch.equal(b[s], d)


# ------------------------------------------------------------------ AdamW
SIZES = (1, 7, 8, 127, 128, 0, 129, 2047, 2048, 2049, 5000)
HYPER = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1)


def _adamw_setup(param, grad, state, rng, sizes=SIZES, grad_std=0.1):
    ps = [draw(rng, n, dtype=F32) for n in sizes]
    masters = [p.clone() for p in ps] if param == "master" else None
    params = ps if param == "f32" else [p.to(BF) for p in ps]
    grads = [draw(rng, n, std=grad_std, dtype=grad) for n in sizes]
    return block.AdamW(params, grads, masters=masters, state=state, seed=77, **HYPER)


@pytest.mark.parametrize("param", ["f32", "bf16", "master"])
@pytest.mark.parametrize("grad", [BF, F32], ids=["gbf16", "gf32"])
def test_adamw_f32_states(param, grad):
    rng = np.random.default_rng(20)
    opt = _adamw_setup(param, grad, "f32", rng)
    at = np.concatenate([[0], np.cumsum([-(-n // 128) * 128 for n in SIZES])])
    gs = torch.tensor(0.5, device=DEV)
    for step in (1, 2, 3):
        old = [f64(p if w is None else w) for p, w in zip(opt.params, opt.masters)]
        om, ov = f64(opt.arena["m"]), f64(opt.arena["v"])
        opt.step(grad_scale=gs if step == 2 else None)
        for i, (p, g, w) in enumerate(zip(opt.params, opt.grads, opt.masters)):
            s = slice(at[i], at[i] + SIZES[i])
            G = f64(g) * (0.5 if step == 2 else 1.0)
            ep, em, ev = OB.adamw(old[i], G, om[s], ov[s], step, 1e-2, 0.9, 0.99, 1e-6, 0.1)
            # a handful of roundings of each term, and of the hyper-parameters
            assert np.all(np.abs(f64(opt.arena["m"][s]) - em) <= 8 * 2.0 ** -24 * (np.abs(om[s]) + np.abs(G)) + 1e-38)
            assert np.all(np.abs(f64(opt.arena["v"][s]) - ev) <= 8 * 2.0 ** -24 * (ov[s] + G * G) + 1e-38)
            bound = 4 * 2.0 ** -24 * np.abs(old[i]) + 64 * 2.0 ** -24 * 0.2 + 1e-38       # |update| < 0.2 here
            if param == "bf16":
                bound = bound + 2 * OB.half_step(ep, 8)
            assert np.all(np.abs(f64(p if w is None else w) - ep) <= bound), (i, step)
            if w is not None:
                assert torch.equal(p, w.to(BF))
    for i in range(len(SIZES)):                                            # between the tensors: untouched
        assert float(opt.arena["m"][at[i] + SIZES[i]:at[i + 1]].abs().sum()) == 0


@pytest.mark.parametrize("param", ["f32", "bf16"])
def test_adamw_8bit_states(param):
    """Codes and scales of every step against the format's definition, from the states before it."""
    rng = np.random.default_rng(21)
    opt = _adamw_setup(param, BF, "q8", rng, sizes=(1, 130, 5, 700))
    sizes, at = (1, 130, 5, 700), [0, 128, 384, 512]
    opt.grads[3][128:256] = 0                                              # a block without gradient
    for step in (1, 2, 3):
        arena = {k: t.cpu().numpy() for k, t in opt.arena.items()}
        val = lambda c, s, signed: OB.code_values(signed)[arena[c].astype(int)] * np.repeat(arena[s].astype(np.float64), 128)
        om, oroot = val("m", "m_scale", True), val("v", "v_scale", False)
        opt.step()
        new = {k: t.cpu().numpy() for k, t in opt.arena.items()}
        off = total = 0
        for i, n in enumerate(sizes):
            G = f64(opt.grads[i])
            pad = -(-n // 128) * 128
            G = np.concatenate([G, np.zeros(pad - n)])
            s = slice(at[i], at[i] + pad)
            m = 0.9 * om[s] + 0.1 * G
            root = np.sqrt(0.99 * oroot[s] ** 2 + 0.01 * G * G)
            for b in range(pad // 128):
                sl = slice(b * 128, b * 128 + 128)
                place = np.arange(at[i] + b * 128, at[i] + b * 128 + 128)
                h = np.array([OB.mixed_bits(j, 77, step) for j in place])
                for x, code, scale, bits, signed in ((m, "m", "m_scale", h >> 13, True),
                                                     (root, "v", "v_scale", ((h * 0x9E3779B1) & 0xFFFFFFFF) >> 13, False)):
                    top = np.abs(x[sl]).max()
                    got = new[scale][(at[i] + b * 128) // 128]
                    assert abs(got - top) <= 8 * 2.0 ** -24 * top
                    want = OB.code_round(x[sl], top, bits, signed)
                    c = new[code][place].astype(int)
                    total += 128
                    off += int((c != want).sum())
                    assert np.all(np.abs((c & 127 if signed else c) - (want & 127 if signed else want)) <= 1)
        # a code differs only where fp32 and exact arithmetic fall on two sides of a random threshold:
        # 2^-21 of a step wide relative to 2^-19 of one, for values up to 32 steps: below 1e-3 of them
        assert off <= max(2, 1e-3 * total), (off, total)
        assert new["m_scale"][(512 + 128) // 128] == 0 and np.all(new["v"][640:768] == 0)


def test_adamw_8bit_states_at_the_ends_of_the_range():
    """Roots far below and above common ones, and a NaN or Inf among a block's gradients, which stays to be seen."""
    sizes = [1e-17, 1e-15, 1e-13, 1.0, 1e18, 1e19]                          # their squares: 1e-34 to 1e38
    g = torch.tensor(sizes, dtype=F32, device=DEV).repeat_interleave(128)
    g = torch.cat([g, torch.ones(256, dtype=F32, device=DEV)])
    g[6 * 128 + 5], g[7 * 128 + 6] = float("nan"), float("inf")
    opt = block.AdamW([torch.zeros_like(g)], [g], lr=1e-3, betas=(0.0, 0.0), eps=1e-30, weight_decay=0.0, state="q8", seed=5)
    opt.step()
    m, r = f64(opt.arena["m_scale"]), f64(opt.arena["v_scale"])
    want = f64(g)[:768:128]
    assert np.all(np.abs(m[:6] - want) <= 2.0 ** -23 * want)
    assert np.all(np.abs(r[:6] - want) <= 2.0 ** -23 * want)               # g g and its root, half a unit each
    assert np.all(opt.arena["v"].cpu().numpy()[:768] >= 254)               # the largest, or one below at a tie
    assert np.isnan(m[6]) and np.isnan(r[6]) and np.isinf(m[7]) and np.isinf(r[7])


def test_adamw_random_rounding_keeps_nan():
    """A NaN of any payload stays one in a parameter that is rounded at random."""
    bits = torch.tensor([0x7FFFFFFF, 0x7FC00000, -1, 0x7F800001], dtype=torch.int32, device=DEV)
    g = bits.repeat(64).view(F32)
    p = torch.ones(g.numel(), dtype=BF, device=DEV)
    opt = block.AdamW([p], [g], lr=1e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.0, seed=1)
    opt.step()
    assert bool(torch.isnan(p).all())


def test_adamw_random_rounding_keeps_small_small_steps():
    """A bf16 parameter without a master moves by a step far below its spacing, on average over elements
    and steps; the mean's deviation is that of independent roundings."""
    n, steps, lr = 1 << 16, 16, 1e-4
    p = torch.full((n,), 1.0, dtype=BF, device=DEV)                        # spacing 2^-8 below 1, 2^-7 above
    g = torch.full((n,), 1.0, dtype=F32, device=DEV)
    opt = block.AdamW([p], [g], lr=lr, betas=(0.0, 0.0), eps=1e-30, weight_decay=0.0, seed=3)
    for _ in range(steps):
        opt.step()
    moved = 1.0 - float(p.double().mean())
    sd = (2.0 ** -8 * lr * steps / n) ** 0.5                               # variance <= spacing * step each time
    assert abs(moved - lr * steps) <= 6 * sd + 1e-7, (moved, lr * steps, sd)
    # the same seed and step: the same bits
    a, b = (torch.full((n,), 1.0, dtype=BF, device=DEV) for _ in range(2))
    for t in (a, b):
        block.AdamW([t], [g], lr=lr, betas=(0.0, 0.0), eps=1e-30, weight_decay=0.0, seed=3).step()
    assert torch.equal(a, b)


def test_adamw_resumes_from_its_arena():
    rng = np.random.default_rng(22)
    a = _adamw_setup("f32", F32, "q8", rng)
    b = block.AdamW([p.clone() for p in a.params], a.grads, state="q8", seed=77, **HYPER)
    a.step()
    b.step()
    c = block.AdamW([p.clone() for p in b.params], a.grads, state="q8", seed=77,
                    arena={k: t.clone() for k, t in b.arena.items()}, **HYPER)
    c.steps = b.steps
    a.step()
    c.step()
    assert all(torch.equal(x, y) for x, y in zip(a.params, c.params))
    assert all(torch.equal(a.arena[k], c.arena[k]) for k in a.arena)


# ------------------------------------------------------------------ streams, graphs, autograd
def test_another_stream():
    rng = np.random.default_rng(30)
    M, H, D = 200, 2, 64
    qkv, do, mod = draw(rng, M, 3 * H * D), draw(rng, M, H, D), draw(rng, 1, H * D)
    pos = torch.arange(M, dtype=torch.int32, device=DEV)[:, None].contiguous()
    norm, rot, att = block.GatedNorm(), block.AxialRotary(D, [D]), block.DocAttention(D)

    def go(stream):
        q, k, v = block.split_qkv(qkv, H, H, D)
        q2, k2 = rot.forward(q, k, pos, stream=stream)
        o, lse = att.forward(q2, k2, v, stream=stream)
        g = att.backward(do, q2, k2, v, o, lse, stream=stream)
        x = o.view(M, H * D)
        r, h, st = norm.forward(x, scale=mod, stream=stream)
        n = norm.backward(h, None, x, None, st, scale=mod, stream=stream)
        return [o, lse, *g, h, n["dx"], n["dscale"]]

    want = go(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        got = go(s)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_graph_replays_match_eager():
    """One step of the operators in a graph, replayed with other work between the replays."""
    rng = np.random.default_rng(31)
    M, H, D = 300, 2, 64
    C = H * D
    x, y = draw(rng, M, C), draw(rng, M, C)
    mod, qkv, pos = draw(rng, 2, 3 * C), draw(rng, M, 3 * C), torch.arange(M, dtype=torch.int32, device=DEV)[:, None].contiguous()
    off = torch.tensor([0, 120, 300], dtype=torch.int32, device=DEV)
    w = draw(rng, D)
    norm, rot, att = block.GatedNorm(), block.AxialRotary(D, [D], q_weight=w, k_weight=w), block.DocAttention(D, mask="causal")

    def step():
        gate, scale, shift = mod.split(C, 1)
        r, h, st = norm.forward(x, y, gate, scale, shift, off)
        q, k, v = block.split_qkv(qkv, H, H, D)
        q2, k2 = rot.forward(q, k, pos)
        o, lse = att.forward(q2, k2, v, off)
        dq, dk, dv = att.backward(h.view(M, H, D), q2, k2, v, o, lse, off)
        g = rot.backward(dq, dk, q, k, pos)
        n = norm.backward(o.view(M, C), r, r, y, st, gate, scale, shift, off)
        return [r, h, o, lse, dv, *g.values(), *[t for t in n.values() if t is not None]]

    ref = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        for t in out:
            t.fill_(0)
        step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, out)), i


def test_autograd_functions():
    """The autograd Functions give the gradients the objects give."""
    rng = np.random.default_rng(32)
    M, H, D = 150, 2, 64
    C = H * D
    leaf = lambda *s: draw(rng, *s).requires_grad_(True)
    x, y, gate, scale, shift, qkv = leaf(M, C), leaf(M, C), leaf(1, C), leaf(1, C), leaf(1, C), leaf(M, 3 * C)
    pos = torch.arange(M, dtype=torch.int32, device=DEV)[:, None].contiguous()
    norm, rot, att = block.GatedNorm(post_norm="rms"), block.AxialRotary(D, [D]), block.DocAttention(D, mask="causal")
    r, h = block.GatedNormFunction.apply(x, y, gate, scale, shift, norm)
    o = block.RotaryAttentionFunction.apply(qkv, pos, rot, att, H, H)
    dr, dh, do = draw(rng, M, C), draw(rng, M, C), draw(rng, M, C)
    torch.autograd.backward([r, h, o], [dr, dh, do])
    with torch.no_grad():
        r2, h2, st = norm.forward(x, y, gate, scale, shift)
        g = norm.backward(dh, dr, r2, y, st, gate, scale, shift)
        q, k, v = block.split_qkv(qkv, H, H, D)
        q2, k2 = rot.forward(q, k, pos)
        o2, lse = att.forward(q2, k2, v)
        dq, dk, dv = att.backward(do.view(M, H, D), q2, k2, v, o2, lse)
        a = rot.backward(dq, dk, q, k, pos)
    assert torch.equal(o, o2.view(M, C)) and torch.equal(h, h2)
    for t, n in ((x, "dx"), (y, "dy"), (gate, "dgate"), (scale, "dscale"), (shift, "dshift")):
        assert torch.equal(t.grad, g[n]), n
    assert torch.equal(qkv.grad, torch.cat([t.reshape(M, C) for t in (a["dq"], a["dk"], dv)], 1))
    # the first norm of a block has no y and no gate; the last step of one no norm
    x2 = leaf(M, C)
    r, h = block.GatedNormFunction.apply(x2, None, None, scale, shift, norm)
    (r.float().sum() + (h * dh).float().sum()).backward()
    assert x2.grad is not None
    r, h = block.GatedNormFunction.apply(x2, y, gate, None, None, norm, None, False)
    assert h is None
    r.backward(dr)
