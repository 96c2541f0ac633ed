"""What a DiT block computes around its quantized linears, and the step that
trains its adapters: objects that hold the weights and plans, allocate
outputs and workspaces with PyTorch, and call the library (the gated residual
and modulated norm, the rotation by positions on several axes, attention
inside packed documents, AdamW over many tensors).  Each has forward and
backward as `layer.QuantizedLinear` has them, and a torch.autograd.Function
for use inside a training graph.

Nothing here computes any part of the operators; it only moves memory and
calls the library.
"""
from __future__ import annotations

import ctypes

import torch

from . import ops

_NORMS = {"none": ops.FT_NORM_NONE, "rms": ops.FT_NORM_RMS, "layer": ops.FT_NORM_LAYER}
_MASKS = {"full": ops.FT_MASK_FULL, "causal": ops.FT_MASK_CAUSAL, "prefix": ops.FT_MASK_PREFIX}
_LAYOUTS = {"pairs": ops.FT_ROPE_PAIRS, "halves": ops.FT_ROPE_HALVES}
_LADDERS = {"axis": ops.FT_ROPE_AXIS, "shared": ops.FT_ROPE_SHARED}
_STATES = {"f32": ops.FT_STATE_F32, "q8": ops.FT_STATE_Q8}
_DTYPES = {torch.bfloat16: ops.FT_BF16, torch.float32: ops.FT_F32}


def _dtype(t: torch.Tensor, what: str) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError(f"{what} must be bfloat16 or float32, not {t.dtype}")
    return _DTYPES[t.dtype]


def _is(t, dtype, what):
    if t is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")


def _shape(t, shape, what):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have the shape {tuple(shape)}, not {tuple(t.shape)}")


def _rows(t, shape, dtype, what):
    """A contiguous tensor of that shape and type, or None."""
    _is(t, dtype, what)
    _shape(t, shape, what)
    if t is not None and not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _head_ld(t: torch.Tensor, heads, dim, what: str) -> int:
    """Row stride of a [M, heads, dim] tensor whose rows hold their heads in one piece."""
    _is(t, torch.bfloat16, what)
    if t.dim() != 3 or t.shape[2] != dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{what} must be [M, {'heads' if heads is None else heads}, {dim}], not {tuple(t.shape)}")
    if t.numel() and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != dim)):
        raise ValueError(f"the heads of a row of {what} must lie next to each other")
    return int(t.stride(0)) if t.shape[0] > 1 else max(int(t.stride(0)), t.shape[1] * dim)


def _offsets(t, what):
    if t is not None:
        _is(t, torch.int32, what)
        if t.dim() != 1 or t.numel() < 2 or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous vector of at least two row offsets")
    return 1 if t is None else int(t.numel()) - 1


class GatedNorm:
    """r = x + alpha * gate_b * (post_weight * N_post(y)),
    h = (1 + scale_b) * (weight * N(r)) + shift_b  (fourtune_norm_fwd / _bwd).

    norm: "layer" or "rms"; post_norm: "none", "rms" or "layer"; weight and
    post_weight: bf16 [C] or None (ones).  The modulation (gate, scale, shift:
    bf16 [samples, C], any row stride, or None) and the samples are arguments
    of each call: `segments` is an int32 device vector of row offsets
    [samples + 1]; without it every sample has M / samples rows."""

    def __init__(self, norm: str = "layer", post_norm: str = "none", weight=None, post_weight=None,
                 eps: float = 1e-6, alpha: float = 1.0):
        self.norm, self.post_norm = _NORMS[norm], _NORMS[post_norm]
        self.weight, self.post_weight = weight, post_weight
        _is(weight, torch.bfloat16, "weight")
        _is(post_weight, torch.bfloat16, "post_weight")
        self.eps, self.alpha = float(eps), float(alpha)
        self._ws = None

    def desc(self, x: torch.Tensor, gate=None, scale=None, shift=None, segments=None) -> ops.FtNorm:
        if x.dim() != 2 or not x.is_contiguous():
            raise ValueError("x must be a contiguous [M, C] tensor")
        M, C = x.shape
        mods = [t for t in (gate, scale, shift) if t is not None]
        n_seg = _offsets(segments, "segments") if segments is not None else (mods[0].shape[0] if mods else 1)
        ld = C
        for t in mods:
            _is(t, torch.bfloat16, "a modulation")
            _shape(t, (n_seg, C), "a modulation")
            if t.stride(1) != 1:
                raise ValueError("a modulation's channels must lie next to each other")
        if mods and n_seg > 1:
            ld = int(mods[0].stride(0))
            if any(t.stride(0) != ld for t in mods):
                raise ValueError("gate, scale and shift must have one row stride")
        for t, what in ((self.weight, "weight"), (self.post_weight, "post_weight")):
            _shape(t, (C,), what)
        p = ops._ptr
        return ops.FtNorm(M, C, n_seg, _dtype(x, "x"), p(segments), self.norm, self.post_norm, self.eps,
                          self.alpha, p(self.weight), p(self.post_weight), p(scale), p(shift), p(gate), ld)

    def forward(self, x, y=None, gate=None, scale=None, shift=None, segments=None, need_h: bool = True,
                stream=None):
        """(r, h, stats); r is x itself without y, h None without need_h."""
        d = self.desc(x, gate, scale, shift, segments)
        _rows(y, x.shape, torch.bfloat16, "y")
        if y is None and not need_h:
            return x, None, None
        r = x if y is None else torch.empty_like(x)
        h = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device) if need_h else None
        stats = torch.empty((x.shape[0], 4), dtype=torch.float32, device=x.device)
        ops.fourtune_norm_fwd(d, x, y, None if y is None else r, h, stats, stream)
        return r, h, stats

    def backward(self, dh, dr, r, y, stats, gate=None, scale=None, shift=None, segments=None,
                 need_weights: bool = True, grad_f32: bool = False, stream=None) -> dict:
        """Gradients by name: dx, dy, dscale, dshift, dgate, dweight,
        dpost_weight; None where there is nothing to differentiate."""
        d = self.desc(r, gate, scale, shift, segments)
        M, C = r.shape
        dev, low = r.device, torch.bfloat16
        _rows(dh, r.shape, low, "dh")
        _rows(dr, r.shape, r.dtype, "dr")
        _rows(y, r.shape, low, "y")
        _rows(stats, (M, 4), torch.float32, "stats")
        gdt = torch.float32 if grad_f32 else low
        mod = lambda t, has: torch.empty((d.n_seg, C), dtype=gdt, device=dev) if t is not None and has else None
        vec = lambda t, has: torch.empty((C,), dtype=gdt, device=dev) if t is not None and has and need_weights else None
        has_h, has_y = dh is not None, y is not None
        g = dict(dx=torch.empty_like(r), dy=torch.empty_like(y) if has_y else None,
                 dscale=mod(scale, has_h), dshift=mod(shift, has_h), dgate=mod(gate, has_y),
                 dweight=vec(self.weight, has_h), dpost_weight=vec(self.post_weight, has_y))
        ws = None
        if any(g[k] is not None for k in ("dscale", "dshift", "dgate", "dweight", "dpost_weight")):
            ws = torch.empty((ops.fourtune_norm_workspace_bytes(d),), dtype=torch.uint8, device=dev)
        ops.fourtune_norm_bwd(d, dh, dr, r, y, stats, g["dx"], g["dy"], g["dscale"], g["dshift"], g["dgate"], C,
                              g["dweight"], g["dpost_weight"], ops.FT_F32 if grad_f32 else ops.FT_BF16, ws,
                              0 if ws is None else ws.numel(), stream)
        return g


class AxialRotary:
    """Rotation of query and key heads by positions on several axes, with an
    optional RMS norm of each head before it (fourtune_rope_fwd / _bwd).

    axis_dims: how many of a head's values each axis rotates, in order;
    layout "pairs" (2j, 2j + 1) or "halves" (j, j + pairs); ladder "axis"
    (every axis its own frequencies) or "shared" (one run divided between the
    axes).  q_weight, k_weight: bf16 [head_dim] of the norms, or None."""

    def __init__(self, head_dim: int, axis_dims, theta: float = 10000.0, layout: str = "pairs",
                 ladder: str = "axis", q_weight=None, k_weight=None, eps: float = 1e-6):
        self.D, self.eps = int(head_dim), float(eps)
        self.table = ops.fourtune_rope_init(self.D, list(axis_dims), theta, _LAYOUTS[layout], _LADDERS[ladder])
        self.n_axes = len(axis_dims)
        self.q_weight, self.k_weight = q_weight, k_weight
        for t, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            _rows(t, (self.D,), torch.bfloat16, what)

    def _side(self, t, out, weight, what):
        return ops.rope_side(t.shape[1], t, out, _head_ld(t, None, self.D, what),
                             _head_ld(out, t.shape[1], self.D, what + "'s output"), weight)

    def forward(self, q, k, positions, q_out=None, k_out=None, stream=None):
        """(q', k'), new [M, heads, D] tensors unless given (which may be q and k
        themselves).  positions: int32 [M, axes]."""
        M = int(q.shape[0])
        _rows(positions, (M, self.n_axes), torch.int32, "positions")
        if k.shape[0] != M:
            raise ValueError("q and k must have the same rows")
        new = lambda t, o: torch.empty(t.shape, dtype=torch.bfloat16, device=t.device) if o is None else o
        q_out, k_out = new(q, q_out), new(k, k_out)
        _shape(q_out, q.shape, "q_out")
        _shape(k_out, k.shape, "k_out")
        ops.fourtune_rope_fwd(self.table, M, positions, self.eps, self._side(q, q_out, self.q_weight, "q"),
                              self._side(k, k_out, self.k_weight, "k"), stream)
        return q_out, k_out

    def backward(self, dq, dk, q, k, positions, dq_out=None, dk_out=None, need_weights: bool = True,
                 grad_f32: bool = False, stream=None) -> dict:
        """Gradients by name: dq, dk, dwq, dwk (the weights', None without
        weights).  dq, dk: of the forward's outputs; q, k: the forward's inputs
        (read where there is a weight); dq_out, dk_out: as in the forward."""
        M = int(dq.shape[0])
        _rows(positions, (M, self.n_axes), torch.int32, "positions")
        new = lambda t, o: torch.empty(t.shape, dtype=torch.bfloat16, device=t.device) if o is None else o
        dq_out, dk_out = new(dq, dq_out), new(dk, dk_out)
        gdt = torch.float32 if grad_f32 else torch.bfloat16
        vec = lambda w, t: torch.empty((self.D,), dtype=gdt, device=dq.device) if w is not None and need_weights and t.shape[1] else None
        dwq, dwk = vec(self.q_weight, dq), vec(self.k_weight, dk)
        xs = []
        for t, g, w, what in ((q, dq, self.q_weight, "q"), (k, dk, self.k_weight, "k")):
            if w is None:
                xs += [None, 0]
            else:
                _shape(t, g.shape, what)
                xs += [t, _head_ld(t, None, self.D, what)]
        ws = None
        if dwq is not None or dwk is not None:
            ws = torch.empty((ops.fourtune_rope_workspace_bytes(self.table, M),), dtype=torch.uint8, device=dq.device)
        ops.fourtune_rope_bwd(self.table, M, positions, self.eps, self._side(dq, dq_out, self.q_weight, "dq"),
                              self._side(dk, dk_out, self.k_weight, "dk"), *xs, dwq, dwk,
                              ops.FT_F32 if grad_f32 else ops.FT_BF16, ws, 0 if ws is None else ws.numel(), stream)
        return dict(dq=dq_out, dk=dk_out, dwq=dwq, dwk=dwk)


class DocAttention:
    """Attention inside packed documents (fourtune_attn_fwd / _bwd).

    mask: "full", "causal" or "prefix"; softcap > 0 caps the scores by a
    tanh; scale defaults to head_dim ** -0.5.  docs: int32 device vector of
    row offsets [documents + 1] (None: one document of all rows); prefix:
    int32 [documents], read by the prefix mask.  q [M, Hq, D], k and v
    [M, Hkv, D] may be parts of one QKV tensor."""

    def __init__(self, head_dim: int, mask: str = "full", softcap: float = 0.0, scale: float | None = None):
        self.D, self.mask, self.softcap = int(head_dim), _MASKS[mask], float(softcap)
        self.scale = self.D ** -0.5 if scale is None else float(scale)

    def desc(self, q, k, v, o, docs=None, prefix=None) -> ops.FtAttn:
        M, Hq, Hkv = int(q.shape[0]), int(q.shape[1]), int(k.shape[1])
        if k.shape[0] != M or v.shape[0] != M:
            raise ValueError("q, k and v must have the same rows")
        n_doc = _offsets(docs, "docs")
        if self.mask == ops.FT_MASK_PREFIX:
            _rows(prefix, (n_doc,), torch.int32, "prefix")
            if prefix is None:
                raise ValueError("the prefix mask needs the prefixes")
        return ops.FtAttn(M, Hq, Hkv, self.D, self.mask, self.scale, self.softcap, n_doc, ops._ptr(docs),
                          ops._ptr(prefix) if self.mask == ops.FT_MASK_PREFIX else None,
                          _head_ld(q, Hq, self.D, "q"), _head_ld(k, Hkv, self.D, "k"),
                          _head_ld(v, Hkv, self.D, "v"), _head_ld(o, Hq, self.D, "o"))

    def forward(self, q, k, v, docs=None, prefix=None, need_lse: bool = True, stream=None):
        """(o [M, Hq, D], lse fp32 [Hq, M])"""
        o = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device) if need_lse else None
        ops.fourtune_attn_fwd(self.desc(q, k, v, o, docs, prefix), q, k, v, o, lse, stream)
        return o, lse

    def backward(self, do, q, k, v, o, lse, docs=None, prefix=None, dq=None, dk=None, dv=None, stream=None):
        """(dq, dk, dv), new tensors unless given (parts of one tensor, say)."""
        new = lambda t, g: torch.empty(t.shape, dtype=torch.bfloat16, device=t.device) if g is None else g
        dq, dk, dv = new(q, dq), new(k, dk), new(v, dv)
        d = self.desc(q, k, v, o, docs, prefix)
        _rows(lse, (q.shape[1], q.shape[0]), torch.float32, "lse")
        ws = torch.empty((ops.fourtune_attn_workspace_bytes(d),), dtype=torch.uint8, device=q.device)
        ld = lambda t, h, what: _head_ld(t, h, self.D, what)
        ops.fourtune_attn_bwd(d, do, ld(do, d.Hq, "do"), q, k, v, o, lse, dq, ld(dq, d.Hq, "dq"), dk,
                              ld(dk, d.Hkv, "dk"), dv, ld(dv, d.Hkv, "dv"), ws, ws.numel(), stream)
        return dq, dk, dv


class AdamW:
    """AdamW over many tensors in one launch (fourtune_adamw_step).

    params: bf16 or fp32 tensors, stepped in place; grads: their gradients
    (bf16 or fp32), fixed tensors that each backward writes into; masters:
    fp32 copies of bf16 params, or None (bf16 params are then rounded at
    random).  state: "f32", or "q8" for states in 8 bits.  `arena` gives
    existing states (m, v, and m_scale, v_scale for q8), as a checkpoint
    holds them."""

    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, masters=None,
                 state: str = "f32", seed: int = 0, arena: dict | None = None):
        params, grads = list(params), list(grads)
        masters = [None] * len(params) if masters is None else list(masters)
        if not params or not len(params) == len(grads) == len(masters):
            raise ValueError("params, grads and masters must be of one length, at least 1")
        for p, g, w in zip(params, grads, masters):
            for t, what in ((p, "a parameter"), (g, "a gradient")) + (((w, "a master"),) if w is not None else ()):
                if not t.is_contiguous() or t.numel() != p.numel() or t.device != params[0].device:
                    raise ValueError(f"{what} must be contiguous, of its parameter's size and on one device")
            _is(w, torch.float32, "a master")
            if p.dtype != params[0].dtype or g.dtype != grads[0].dtype:
                raise TypeError("the parameters must be of one type, and so the gradients")
        self.params, self.grads, self.masters = params, grads, masters
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.seed, self.steps = int(seed), 0
        dev = params[0].device
        n = len(params)
        table = (ops.FtAdamwTensor * n)(*[ops.FtAdamwTensor(ops._ptr(p), ops._ptr(g), ops._ptr(w), p.numel())
                                          for p, g, w in zip(params, grads, masters)])
        size, total = ops.fourtune_adamw_plan_bytes(table, n)
        host = torch.empty((max(size, 1),), dtype=torch.uint8)
        self.desc = ops.fourtune_adamw_plan(table, n, _dtype(params[0], "a parameter"), _dtype(grads[0], "a gradient"),
                                            _STATES[state], host, host.numel())
        self.table = host.to(dev)
        q8 = state == "q8"
        kinds = dict(m=(total, torch.uint8 if q8 else torch.float32), v=(total, torch.uint8 if q8 else torch.float32))
        if q8:
            kinds.update(m_scale=(total // 128, torch.float32), v_scale=(total // 128, torch.float32))
        self.arena = {}
        for k, (size, dtype) in kinds.items():
            t = torch.zeros((size,), dtype=dtype, device=dev) if arena is None else arena[k]
            _rows(t, (size,), dtype, k)
            self.arena[k] = t
            setattr(self.desc, k, ops._ptr(t))
        self.desc.table = ops._ptr(self.table)

    def step(self, grad_scale=None, stream=None):
        """One step; grad_scale: an fp32 device scalar that multiplies every
        gradient (a clipping factor), or None."""
        _is(grad_scale, torch.float32, "grad_scale")
        self.steps += 1
        ops.fourtune_adamw_step(self.desc, self.steps, self.lr, *self.betas, self.eps, self.weight_decay, self.seed,
                                grad_scale, stream)


class GatedNormFunction(torch.autograd.Function):
    """(r, h) = norm(x, y, gate, scale, shift) with gradients for all five (the
    norm's weights are frozen here)."""

    @staticmethod
    def forward(ctx, x, y, gate, scale, shift, norm: GatedNorm, segments=None, need_h: bool = True):
        r, h, stats = norm.forward(x, y, gate, scale, shift, segments, need_h)
        ctx.norm, ctx.segments = norm, segments
        ctx.save_for_backward(r, y, gate, scale, shift, stats)
        if r is x:
            r = x.view_as(x)
        return r, h

    @staticmethod
    def backward(ctx, dr, dh):
        r, y, gate, scale, shift, stats = ctx.saved_tensors
        if dh is None and y is None:
            return (dr,) + (None,) * 7
        g = ctx.norm.backward(None if dh is None else dh.contiguous(), None if dr is None else dr.contiguous(), r, y,
                              stats, gate, scale, shift, ctx.segments, need_weights=False)
        return g["dx"], g["dy"], g["dgate"], g["dscale"], g["dshift"], None, None, None


class RotaryAttentionFunction(torch.autograd.Function):
    """o = attention(rotate(q), rotate(k), v) of a fused QKV tensor [M, (Hq + 2
    Hkv) D], with its gradient written as one tensor of the same layout."""

    @staticmethod
    def forward(ctx, qkv, positions, rope: AxialRotary, attn: DocAttention, Hq: int, Hkv: int, docs=None, prefix=None):
        q, k, v = split_qkv(qkv, Hq, Hkv, attn.D)
        q2, k2 = rope.forward(q, k, positions)
        o, lse = attn.forward(q2, k2, v, docs, prefix)
        ctx.plan = (rope, attn, Hq, Hkv, docs, prefix)
        ctx.save_for_backward(qkv, positions, q2, k2, o, lse)
        return o.view(o.shape[0], -1)

    @staticmethod
    def backward(ctx, do):
        rope, attn, Hq, Hkv, docs, prefix = ctx.plan
        qkv, positions, q2, k2, o, lse = ctx.saved_tensors
        q, k, v = split_qkv(qkv, Hq, Hkv, attn.D)
        dqkv = torch.empty_like(qkv)
        dq, dk, dv = split_qkv(dqkv, Hq, Hkv, attn.D)
        attn.backward(do.contiguous().view(o.shape), q2, k2, v, o, lse, docs, prefix, dq, dk, dv)
        rope.backward(dq, dk, q, k, positions, dq, dk, need_weights=False)
        return (dqkv,) + (None,) * 7


def split_qkv(qkv: torch.Tensor, Hq: int, Hkv: int, D: int):
    """Views [M, heads, D] of the queries, keys and values of a fused row."""
    q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], 1)
    return q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D))
