"""C-ABI checks of the operators around the linears that need no GPU: every
bad argument is refused on the host before anything is read (fake addresses
are never dereferenced), and the Python objects refuse wrong tensors."""
import ctypes
import os

import pytest
import torch

from bit_quantized_amd import block, ops

pytestmark = pytest.mark.skipif(not os.path.exists(ops.LIB_PATH), reason="libfourtune.so not built")
A = 0x10000000      # a fake 16-byte-aligned device address
BIG = 1 << 40
OK = ops.FT_EUNSUPPORTED    # only the missing GPU stops a good call here


def norm(**kw):
    d = dict(M=10, C=64, n_seg=2, stream_dtype=ops.FT_BF16, seg=A, norm=ops.FT_NORM_LAYER, post_norm=ops.FT_NORM_RMS,
             eps=1e-6, alpha=1.0, weight=A, post_weight=A, scale=A, shift=A, gate=A, ld_mod=64)
    d.update(kw)
    return ops.FtNorm(**d)


def norm_fwd(d, x=A, y=A, r=A, h=A, stats=A):
    return ops.lib().fourtune_norm_fwd(ctypes.byref(d), x, y, r, h, stats, None)


def norm_bwd(d, dh=A, dr=A, r=A, y=A, stats=A, dx=A, dy=A, ds=A, dsh=A, dg=A, ld=64, dw=A, dpw=A, gdt=0, ws=A, wsb=BIG):
    return ops.lib().fourtune_norm_bwd(ctypes.byref(d), dh, dr, r, y, stats, dx, dy, ds, dsh, dg, ld, dw, dpw, gdt, ws,
                                       wsb, None)


def test_norm_refusals():
    assert norm_fwd(norm()) == OK and norm_bwd(norm()) == OK
    for kw in (dict(M=-1), dict(C=4), dict(C=60), dict(C=16392), dict(n_seg=0), dict(n_seg=1 << 20),
               dict(seg=None, M=11)):
        assert norm_fwd(norm(**kw)) == ops.FT_ESHAPE, kw
        assert norm_bwd(norm(**kw)) == ops.FT_ESHAPE, kw
        assert ops.fourtune_norm_workspace_bytes(norm(**kw)) == 0
    for kw in (dict(stream_dtype=2), dict(norm=0), dict(norm=3), dict(post_norm=-1), dict(eps=-1.0),
               dict(eps=float("nan")), dict(alpha=float("inf"))):
        assert norm_fwd(norm(**kw)) == ops.FT_EINVAL, kw
    for kw in (dict(ld_mod=56), dict(ld_mod=68), dict(weight=A + 2), dict(gate=A + 8), dict(scale=A + 4), dict(seg=A + 2)):
        assert norm_fwd(norm(**kw)) == ops.FT_EALIGN, kw
    assert norm_fwd(norm(), x=None) == ops.FT_EINVAL
    assert norm_fwd(norm(), r=None) == ops.FT_EINVAL                      # y needs somewhere to go
    assert norm_fwd(norm(), y=None, r=None, h=None) == ops.FT_EINVAL      # nothing asked for
    assert norm_fwd(norm(), x=A + 8) == ops.FT_EALIGN
    assert norm_fwd(norm(gate=A + 8, post_norm=9), y=None) == OK          # not read without y
    assert norm_fwd(norm(norm=9, weight=A + 2), h=None) == OK             # not read without h
    assert norm_fwd(norm(M=0), x=None, y=None, r=None, h=None, stats=None) == ops.FT_OK
    assert norm_bwd(norm(), dx=None) == ops.FT_EINVAL
    assert norm_bwd(norm(), dy=None) == ops.FT_EINVAL
    assert norm_bwd(norm(), stats=None) == ops.FT_EINVAL
    assert norm_bwd(norm(), dh=None, y=None, ds=None, dsh=None, dg=None, dw=None, dpw=None) == ops.FT_EINVAL
    assert norm_bwd(norm(), dh=None) == ops.FT_EINVAL                     # dscale needs dh
    assert norm_bwd(norm(), y=None) == ops.FT_EINVAL                      # dgate needs y
    assert norm_bwd(norm(), gdt=5) == ops.FT_EINVAL
    assert norm_bwd(norm(), ld=60) == ops.FT_EALIGN
    need = ops.fourtune_norm_workspace_bytes(norm())
    assert norm_bwd(norm(), wsb=need - 1) == ops.FT_EWORKSPACE and norm_bwd(norm(), wsb=need) == OK
    assert norm_bwd(norm(), ws=None) == ops.FT_EINVAL
    assert norm_bwd(norm(), ws=None, wsb=0, ds=None, dsh=None, dg=None, dw=None, dpw=None) == OK


def rope(D=64, dims=(32, 32), theta=1e4, layout=0, ladder=0):
    rp = ops.FtRope()
    s = ops.lib().fourtune_rope_init(ctypes.byref(rp), D, len(dims), (ctypes.c_int32 * len(dims))(*dims), theta, layout, ladder)
    return s, rp


def side(heads=2, inp=A, out=A, ld_in=128, ld_out=128, weight=A):
    return ops.FtRopeSide(heads, inp, out, ld_in, ld_out, weight)


def rope_fwd(rp, M=5, pos=A, eps=1e-6, q=None, k=None):
    return ops.lib().fourtune_rope_fwd(ctypes.byref(rp), M, pos, eps, ctypes.byref(q or side()), ctypes.byref(k or side()), None)


def rope_bwd(rp, M=5, pos=A, q=None, k=None, qx=A, ldq=128, kx=A, ldk=128, dqw=A, dkw=A, gdt=0, ws=A, wsb=BIG):
    return ops.lib().fourtune_rope_bwd(ctypes.byref(rp), M, pos, 1e-6, ctypes.byref(q or side()), ctypes.byref(k or side()),
                                       qx, ldq, kx, ldk, dqw, dkw, gdt, ws, wsb, None)


def test_rope_refusals():
    for kw in (dict(D=60), dict(D=264), dict(D=0), dict(dims=(32, 34)), dict(dims=(31,)), dict(dims=(0, 2)),
               dict(dims=(12, 12, 12, 12, 12)), dict(layout=1, dims=(24,))):
        assert rope(**kw)[0] == ops.FT_ESHAPE, kw
    for kw in (dict(theta=0.0), dict(theta=float("inf")), dict(layout=2), dict(ladder=-1)):
        assert rope(**kw)[0] == ops.FT_EINVAL, kw
    s, rp = rope()
    assert s == ops.FT_OK and rope_fwd(rp) == OK and rope_bwd(rp) == OK
    assert rope_fwd(ops.FtRope()) == ops.FT_ESHAPE                        # never filled
    bad = ops.FtRope.from_buffer_copy(rp)
    bad.axis[3] = 2
    assert rope_fwd(bad) == ops.FT_EINVAL
    assert rope_fwd(rp, M=-1) == ops.FT_ESHAPE and rope_fwd(rp, M=0, pos=None) == ops.FT_OK
    assert rope_fwd(rp, pos=None) == ops.FT_EINVAL and rope_fwd(rp, eps=-1.0) == ops.FT_EINVAL
    assert rope_fwd(rp, pos=A + 2) == ops.FT_EALIGN
    assert rope_fwd(rp, q=side(heads=-1)) == ops.FT_ESHAPE
    assert rope_fwd(rp, q=side(heads=0, inp=None, out=None), k=side(heads=0, inp=None, out=None)) == ops.FT_OK
    assert rope_fwd(rp, k=side(inp=None)) == ops.FT_EINVAL and rope_fwd(rp, k=side(out=None)) == ops.FT_EINVAL
    assert rope_fwd(rp, q=side(ld_in=120)) == ops.FT_EALIGN and rope_fwd(rp, q=side(ld_out=132)) == ops.FT_EALIGN
    assert rope_fwd(rp, q=side(ld_in=136)) == ops.FT_EINVAL               # in place with two strides
    assert rope_fwd(rp, q=side(weight=A + 2)) == ops.FT_EALIGN
    assert rope_bwd(rp, qx=None) == ops.FT_EINVAL and rope_bwd(rp, ldk=120) == ops.FT_EALIGN
    assert rope_bwd(rp, q=side(weight=None)) == ops.FT_EINVAL             # a gradient of no weight
    assert rope_bwd(rp, q=side(weight=None), dqw=None, qx=None) == OK
    assert rope_bwd(rp, gdt=9) == ops.FT_EINVAL
    need = ops.fourtune_rope_workspace_bytes(rp, 5)
    assert rope_bwd(rp, wsb=need - 1) == ops.FT_EWORKSPACE and rope_bwd(rp, ws=None) == ops.FT_EINVAL
    assert rope_bwd(rp, ws=None, wsb=0, dqw=None, dkw=None) == OK


def attn(**kw):
    d = dict(M=100, Hq=4, Hkv=2, D=64, mask=ops.FT_MASK_PREFIX, scale=0.1, softcap=0.0, n_doc=3, doc=A, prefix=A, ld_q=256,
             ld_k=128, ld_v=128, ld_o=256)
    d.update(kw)
    return ops.FtAttn(**d)


def attn_fwd(d, q=A, k=A, v=A, o=A, lse=A):
    return ops.lib().fourtune_attn_fwd(ctypes.byref(d), q, k, v, o, lse, None)


def attn_bwd(d, do=A, ldo=256, q=A, k=A, v=A, o=A, lse=A, dq=A, lq=256, dk=A, lk=128, dv=A, lv=128, ws=A, wsb=BIG):
    return ops.lib().fourtune_attn_bwd(ctypes.byref(d), do, ldo, q, k, v, o, lse, dq, lq, dk, lk, dv, lv, ws, wsb, None)


def test_attention_grid_limit():
    """Documents times heads have to fit one grid of workgroups."""
    assert attn_fwd(attn(n_doc=(1 << 20) - 3)) == OK and attn_bwd(attn(n_doc=(1 << 20) - 3)) == OK
    assert attn_fwd(attn(n_doc=(1 << 20) - 2)) == ops.FT_ESHAPE
    assert attn_bwd(attn(n_doc=(1 << 20) - 2)) == ops.FT_ESHAPE


def test_attention_refusals():
    assert attn_fwd(attn()) == OK and attn_bwd(attn()) == OK
    for kw in (dict(M=-1), dict(D=96), dict(D=32), dict(Hq=0), dict(Hkv=0), dict(Hkv=3), dict(n_doc=0), dict(doc=None),
               dict(n_doc=1 << 21), dict(ld_k=1 << 23), dict(M=1 << 30, Hq=1024, ld_q=1 << 16, ld_o=1 << 16)):
        assert attn_fwd(attn(**kw)) == ops.FT_ESHAPE, kw
        assert attn_bwd(attn(**kw)) == ops.FT_ESHAPE, kw
    for kw in (dict(mask=3), dict(mask=-1), dict(prefix=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(softcap=-1.0), dict(softcap=float("inf"))):
        assert attn_fwd(attn(**kw)) == ops.FT_EINVAL, kw
    for kw in (dict(ld_q=248), dict(ld_k=132), dict(ld_v=120), dict(ld_o=0), dict(doc=A + 2), dict(prefix=A + 1)):
        assert attn_fwd(attn(**kw)) == ops.FT_EALIGN, kw
    assert attn_fwd(attn(mask=ops.FT_MASK_CAUSAL, prefix=None)) == OK
    assert attn_fwd(attn(doc=None, n_doc=1)) == OK
    assert attn_fwd(attn(), lse=None) == OK
    for name in "qkvo":
        assert attn_fwd(attn(), **{name: None}) == ops.FT_EINVAL
        assert attn_fwd(attn(), **{name: A + 8}) == ops.FT_EALIGN
    assert attn_fwd(attn(M=0), q=None, k=None, v=None, o=None, lse=None) == ops.FT_OK
    for name in ("do", "lse", "dq", "dk", "dv", "o"):
        assert attn_bwd(attn(), **{name: None}) == ops.FT_EINVAL
    for name in ("ldo", "lq", "lk", "lv"):
        assert attn_bwd(attn(), **{name: 60}) == ops.FT_EALIGN
    need = ops.fourtune_attn_workspace_bytes(attn())
    assert attn_bwd(attn(), wsb=need - 1) == ops.FT_EWORKSPACE and attn_bwd(attn(), wsb=need) == OK
    assert attn_bwd(attn(), ws=None) == ops.FT_EINVAL
    assert ops.fourtune_attn_workspace_bytes(attn(D=48)) == 0


def _plan(ts, pd=ops.FT_BF16, gd=ops.FT_BF16, st=ops.FT_STATE_F32, short=0):
    arr = (ops.FtAdamwTensor * len(ts))(*[ops.FtAdamwTensor(*t) for t in ts])
    size, _ = ops.fourtune_adamw_plan_bytes(arr, len(ts))
    host = (ctypes.c_uint8 * max(size, 1))()
    d = ops.FtAdamw()
    s = ops.lib().fourtune_adamw_plan(arr, len(ts), pd, gd, st, ctypes.byref(d), ctypes.addressof(host), size - short)
    return s, d


def _step(d, t=1, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, gs=None):
    return ops.lib().fourtune_adamw_step(ctypes.byref(d), t, lr, b1, b2, eps, wd, 1, gs, None)


def test_adamw_refusals():
    one = (A, A, None, 100)
    s, d = _plan([one, (None, None, None, 0)])
    assert s == ops.FT_OK
    d.table, d.m, d.v = A, A, A
    assert _step(d) == OK
    assert _plan([one], short=1)[0] == ops.FT_EWORKSPACE
    assert _plan([(A, A, None, -1)])[0] == ops.FT_ESHAPE
    assert _plan([(A, A, None, 1 << 31), (A, A, None, 1 << 31)])[0] == ops.FT_ESHAPE     # arena of 2^32
    assert _plan([(None, A, None, 5)])[0] == ops.FT_EINVAL and _plan([(A, None, None, 5)])[0] == ops.FT_EINVAL
    assert _plan([(A + 2, A, None, 5)])[0] == ops.FT_EALIGN and _plan([(A, A, A + 4, 5)])[0] == ops.FT_EALIGN
    assert _plan([one, (A, A, A, 5)])[0] == ops.FT_EINVAL                                # masters of some
    assert _plan([(A, A, A, 5)], pd=ops.FT_F32)[0] == ops.FT_EINVAL                      # a master of fp32
    assert _plan([one], pd=7)[0] == ops.FT_EINVAL and _plan([one], gd=-1)[0] == ops.FT_EINVAL
    assert _plan([one], st=2)[0] == ops.FT_EINVAL
    for kw in (dict(t=0), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(eps=0.0), dict(lr=float("nan")),
               dict(wd=float("inf"))):
        assert _step(d, **kw) == ops.FT_EINVAL, kw
    assert _step(d, gs=A + 2) == ops.FT_EALIGN
    d.m = None
    assert _step(d) == ops.FT_EINVAL
    s, q = _plan([one], st=ops.FT_STATE_Q8)
    q.table, q.m, q.v = A, A, A
    assert s == ops.FT_OK and _step(q) == ops.FT_EINVAL                                  # the scales are missing
    q.m_scale, q.v_scale = A, A + 4
    assert _step(q) == ops.FT_EALIGN
    s, empty = _plan([(None, None, None, 0)])
    assert s == ops.FT_OK and _step(empty) == ops.FT_OK                                  # nothing to do


def test_objects_refuse_wrong_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    n = block.GatedNorm(norm="rms", weight=bf(16))
    with pytest.raises(ValueError):
        n.forward(bf(4, 32).t())
    with pytest.raises(ValueError):
        n.forward(torch.zeros(4, 16, dtype=torch.float16))
    with pytest.raises(ValueError):
        n.forward(bf(4, 32))                                              # the weight has 16 channels
    with pytest.raises(ValueError):
        n.forward(bf(4, 16), scale=bf(2, 8))
    with pytest.raises(ValueError):
        n.forward(bf(4, 16), scale=bf(2, 16), shift=bf(2, 32)[:, :16])    # two strides
    with pytest.raises(TypeError):
        n.forward(bf(4, 16), segments=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        n.forward(bf(4, 16), y=torch.zeros(4, 16))
    with pytest.raises(KeyError):
        block.GatedNorm(norm="batch")
    r = block.AxialRotary(16, [8, 8])
    with pytest.raises(ValueError):
        r.forward(bf(4, 2, 32), bf(4, 2, 16), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        r.forward(bf(4, 2, 16), bf(4, 2, 16), torch.zeros(4, 2))
    with pytest.raises(ValueError):
        r.forward(bf(4, 2, 16), bf(3, 2, 16), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ops.FourTuneError):
        block.AxialRotary(16, [8, 16])
    a = block.DocAttention(64, mask="prefix")
    with pytest.raises(ValueError):
        a.forward(bf(4, 2, 64), bf(4, 2, 64), bf(4, 2, 64))               # no prefixes
    with pytest.raises(ValueError):
        block.DocAttention(64).forward(bf(4, 2, 64), bf(5, 2, 64), bf(4, 2, 64))
    with pytest.raises(ValueError):
        block.DocAttention(64).forward(bf(4, 64, 2).transpose(1, 2), bf(4, 2, 64), bf(4, 2, 64))
    with pytest.raises(TypeError):
        block.AdamW([bf(8), torch.zeros(8)], [bf(8), bf(8)])
    with pytest.raises(ValueError):
        block.AdamW([bf(8)], [bf(9)])
    with pytest.raises(ValueError):
        block.AdamW([], [])
