"""Cases of the operators around the quantized linears of a DiT block, and their plain forms.

The quantized linears of a block under 4-bit post-training leave four kinds of work between them and after them:

  norm   the gated residual of one sub-block and the modulated norm before the next, per sample of the batch
  rope   the per-head RMS norm of queries and keys and their rotation by positions on several axes
  attn   attention inside packed documents, optionally behind a prefix and with scores capped by a tanh
  adamw  the step of the adapters' optimizer, states in 32 bits or in 8

`listed()` holds the sizes of a step, `draw()` gives more of the same ranges, `run()` computes one case in its plain form
(elementary torch operations in 32 bits) or, where `own` is true, with the package's operators.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the modulated norm in front of the fused QKV linear, one 1024x1024 image with its text, while sampling
        dict(name="norm_sample", op="norm", train=False, rows="4608", chan=3072, norm="layer", post="none", gated=False,
             stream="bf16"),
        # a training step at batch 2: attention's output gated into the stream, then the MLP's modulated norm
        dict(name="norm_gate_train", op="norm", train=True, rows="4608,4608", chan=3072, norm="layer", post="none",
             gated=True, stream="bf16"),
        # samples of unequal length, norms before and after the sub-block with weights, the stream kept in 32 bits
        dict(name="norm_sandwich_ragged", op="norm", train=True, rows="1,837,0,703", chan=1160, norm="rms", post="rms",
             gated=True, stream="f32"),
        # the text encoder's side of a small step: one rotation without norms, 77 tokens, halves layout
        dict(name="rope_text", op="rope", train=False, tokens=77, hq=12, hkv=12, dim=64, axes="64", layout="halves",
             ladder="axis", normed=False),
        # image and text tokens of the QKV linear's output, three axes, with its gradient
        dict(name="rope_qkv_train", op="rope", train=True, tokens=4608, hq=24, hkv=24, dim=128, axes="16,56,56",
             layout="pairs", ladder="axis", normed=True),
        # a video clip: time, height and width share one ladder of frequencies, fewer key heads than query heads
        dict(name="rope_video", op="rope", train=False, tokens=16380, hq=16, hkv=4, dim=128, axes="32,48,48",
             layout="halves", ladder="shared", normed=True),
        # the attention of one sampling step, text and image tokens together
        dict(name="attn_image", op="attn", train=False, docs="4608", outside=0, hq=24, hkv=24, dim=128, mask="full",
             cap=0.0),
        # a training step at batch 2, the two samples packed
        dict(name="attn_train", op="attn", train=True, docs="4608,4608", outside=0, hq=24, hkv=24, dim=128, mask="full",
             cap=0.0),
        # many documents in one row of a pretraining batch, some empty or of one token, prompt prefixes, capped scores
        dict(name="attn_packed_train", op="attn", train=True, docs="1,640,0,77,513,1024,2,435", outside=19, hq=12, hkv=4,
             dim=64, mask="prefix", cap=30.0),
        # one layer's adapter: the smallest step there is
        dict(name="adamw_layer", op="adamw", state="f32", param="f32", shapes="16x257,16x1000", copies=1),
        # every adapter of the linears of 16 double-stream blocks (rank 16): 320 tensors, 32-bit states and masters
        dict(name="adamw_blocks", op="adamw", state="f32", param="master", copies=32,
             shapes="16x3072,16x9216,16x3072,16x3072,16x3072,16x12288,16x12288,16x3072,16x3072,16x18432"),
        # the same at rank 64 without the modulation, states in 8 bits and no masters
        dict(name="adamw_blocks_8bit", op="adamw", state="q8", param="bf16", copies=32,
             shapes="64x3072,64x9216,64x3072,64x3072,64x3072,64x12288,64x12288,64x3072"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cut(rng, total, parts):
    """`total` in so many parts, some of them small."""
    at = sorted(rng.randint(0, total) for _ in range(parts - 1))
    return [b - a for a, b in zip([0] + at, at + [total])]


def draw(rng):
    op = rng.choice(["norm", "rope", "attn", "adamw"])
    if op == "norm":
        chan = 8 * _log(rng, 16, 1536)
        total = _log(rng, 1, max(2, min(9216, 28_000_000 // chan)))
        rows = _cut(rng, total, rng.choice([1, 1, 2, 3, 8]))
        post = rng.choice(["none", "none", "rms", "layer"])
        return dict(op=op, train=rng.random() < 0.6, rows=",".join(map(str, rows)), chan=chan, norm=rng.choice(["layer", "rms"]),
                    post=post, gated=post != "none" or rng.random() < 0.6, stream=rng.choice(["bf16", "f32"]))
    if op == "rope":
        layout = rng.choice(["pairs", "halves"])
        dim = rng.choice([64, 128, 128, 96, 72] if layout == "pairs" else [64, 128, 128, 96])
        hkv = rng.choice([1, 2, 4, 8, 12, 24])
        hq = hkv * rng.choice([1, 1, 2, 3, 4] if hkv <= 8 else [1, 2])
        unit = 2 if layout == "pairs" else 16
        left, axes = dim // unit, []
        for _ in range(rng.choice([1, 2, 3, 3]) - 1):
            take = rng.randint(1, max(1, left // 2))
            axes, left = axes + [take * unit], left - take
        axes.append(left * unit)
        tokens = _log(rng, 1, max(2, min(16384, 56_000_000 // ((hq + hkv) * dim))))
        return dict(op=op, train=rng.random() < 0.6, tokens=tokens, hq=hq, hkv=hkv, dim=dim, axes=",".join(map(str, axes)),
                    layout=layout, ladder=rng.choice(["axis", "shared"]), normed=rng.random() < 0.6)
    if op == "attn":
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4])
        docs = _cut(rng, _log(rng, 1, 4096 if hq > 12 else 6144), rng.choice([1, 1, 2, 5, 16]))
        return dict(op=op, train=rng.random() < 0.6, docs=",".join(map(str, docs)), outside=rng.choice([0, 0, 1, 50]), hq=hq, hkv=hkv,
                    dim=rng.choice([64, 128]), mask=rng.choice(["full", "prefix", "causal"]), cap=rng.choice([0.0, 0.0, 30.0, 50.0]))
    shapes = ["%dx%d" % (rng.choice([1, 4, 8, 16, 32, 64]), _log(rng, 1, 16000)) for _ in range(rng.randint(1, 10))]
    return dict(op=op, state=rng.choice(["f32", "q8"]), param=rng.choice(["f32", "bf16", "master"]), shapes=",".join(shapes),
                copies=_log(rng, 1, 8))


def _ints(text):
    return [int(t) for t in str(text).split(",")]


def _sizes(case):
    one = [int(a) * int(b) for a, b in (t.split("x") for t in case["shapes"].split(","))]
    return one * case["copies"]


def _prefixes(case):
    """Keys of each document that every query of it sees: a quarter of it where there is a prefix mask."""
    return [n // 4 if case["mask"] == "prefix" else 0 for n in _ints(case["docs"])]


def _pairs(case):
    if case["mask"] == "full":
        return sum(n * n for n in _ints(case["docs"]))
    return sum(n * (n + 1) // 2 + p * (p - 1) // 2 * (p > 0) for n, p in zip(_ints(case["docs"]), _prefixes(case)))


def work(case):
    op = case["op"]
    if op == "norm":
        n, s = sum(_ints(case["rows"])) * case["chan"], 2 if case["stream"] == "bf16" else 4
        y, train = case["gated"], case["train"]
        by = n * (s + 2) + (n * (2 + s) if y else 0)                    # x, h; y, r
        by += n * (2 + 2 * s) + (n * 2 if y else 0) if train else 0       # dh, dr, dx; dy
        return dict(bytes=by, flops=n * (8 + 4 * y + (16 + 6 * y) * train))
    if op == "rope":
        n = case["tokens"] * (case["hq"] + case["hkv"]) * case["dim"]
        return dict(bytes=n * (8 if case["train"] else 4) + case["tokens"] * 4 * len(_ints(case["axes"])),
                    flops=n * (6 + 14 * case["train"]))
    if op == "attn":
        t, d = sum(_ints(case["docs"])) + case["outside"], case["dim"]
        q, k = t * case["hq"] * d * 2, t * case["hkv"] * d * 2
        return dict(bytes=2 * q + 2 * k + t * case["hq"] * 4 + (2 * q + 2 * k) * case["train"],
                    flops=(14 if case["train"] else 4) * d * case["hq"] * _pairs(case))
    n = sum(_sizes(case))
    by = {"f32": 8 + 2, "bf16": 4 + 2, "master": 8 + 2 + 2}[case["param"]] + (16 if case["state"] == "f32" else 4 + 16 / 128)
    return dict(bytes=n * by, flops=n * 20)


# ------------------------------------------------------------------------------------------------- inputs
class _Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)

    def n(self, *shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=self.g, device=DEV) * std).to(dtype)

    def i(self, lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=self.g, device=DEV, dtype=torch.int32)


def _offsets(lengths, first=0):
    at = [first]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    return {"norm": _prepare_norm, "rope": _prepare_rope, "attn": _prepare_attn, "adamw": _prepare_adamw}[case["op"]](case, _Draw(seed))


def _prepare_norm(case, d):
    rows, c = _ints(case["rows"]), case["chan"]
    m, b = sum(rows), len(rows)
    dtype = torch.bfloat16 if case["stream"] == "bf16" else torch.float32
    loud = 1 + 9 * (torch.rand(c, generator=d.g, device=DEV) < 0.01)                 # some channels are ten times louder
    s = dict(case=case, x=(d.n(m, c, dtype=torch.float32) * loud + 0.1).to(dtype), seg=_offsets(rows))
    s["mod"] = d.n(b, 3 * c, std=0.3)                                                # the modulation linear's output
    if case["gated"]:
        s["y"] = d.n(m, c, std=0.7)
    if case["norm"] == "rms":
        s["weight"] = (1 + d.n(c, std=0.1, dtype=torch.float32)).to(torch.bfloat16)
    if case["post"] == "rms":
        s["post_weight"] = (1 + d.n(c, std=0.1, dtype=torch.float32)).to(torch.bfloat16)
    if case["train"]:
        s["dh"], s["dr"] = d.n(m, c, std=1e-3), d.n(m, c, std=1e-3, dtype=dtype)
    if own:
        from bit_quantized_amd import block
        s["op"] = block.GatedNorm(norm=case["norm"], post_norm=case["post"], weight=s.get("weight"),
                                  post_weight=s.get("post_weight"), eps=1e-6)
    return s


def _prepare_rope(case, d):
    m, hq, hkv, dim = case["tokens"], case["hq"], case["hkv"], case["dim"]
    axes = _ints(case["axes"])
    side = max(1, math.isqrt(m))
    t = torch.arange(m, device=DEV, dtype=torch.int32)
    every = [t, t // side, t % side] if len(axes) == 1 else [t // (side * 16), t // side, t % side]
    s = dict(case=case, pos=torch.stack(every[:len(axes)], 1).contiguous() + d.i(0, 50, 1), qkv=d.n(m, (hq + 2 * hkv) * dim))
    if case["normed"]:
        s["wq"], s["wk"] = ((1 + d.n(dim, std=0.1, dtype=torch.float32)).to(torch.bfloat16) for _ in range(2))
    if case["train"]:
        s["dq"], s["dk"] = d.n(m, hq, dim, std=1e-3), d.n(m, hkv, dim, std=1e-3)
    if own:
        from bit_quantized_amd import block
        s["op"] = block.AxialRotary(dim, axes, theta=10000.0, layout=case["layout"], ladder=case["ladder"],
                                    q_weight=s.get("wq"), k_weight=s.get("wk"), eps=1e-6)
    return s


def _prepare_attn(case, d):
    docs, hq, hkv, dim = _ints(case["docs"]), case["hq"], case["hkv"], case["dim"]
    first = case["outside"] // 3
    m = sum(docs) + case["outside"]
    s = dict(case=case, q=d.n(m, hq, dim, std=1.3), k=d.n(m, hkv, dim, std=1.3), qkv=d.n(m, (hq + 2 * hkv) * dim),
             docs=_offsets(docs, first), prefix=torch.tensor(_prefixes(case), dtype=torch.int32, device=DEV), first=first)
    if case["train"]:
        s["do"] = d.n(m, hq, dim, std=1e-3)
    if own:
        from bit_quantized_amd import block
        s["op"] = block.DocAttention(dim, mask=case["mask"], softcap=case["cap"])
    return s


HYPER = dict(lr=3e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01)


def _prepare_adamw(case, d):
    sizes = _sizes(case)
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // 128) * 128)                                       # each tensor starts on a block
    total = at[-1]
    inside = torch.zeros(total, dtype=torch.bool, device=DEV)
    for a, n in zip(at, sizes):
        inside[a:a + n] = True
    loud = torch.exp(d.n(total // 128, 1, std=1.0, dtype=torch.float32)).expand(-1, 128).reshape(-1)
    p = d.n(total, std=0.02, dtype=torch.float32) * inside
    g = (d.n(total, std=1e-3, dtype=torch.float32) * loud * inside).to(torch.float32 if case["param"] == "f32" else torch.bfloat16)
    m = d.n(total, std=3e-4, dtype=torch.float32) * loud * inside
    v = (d.n(total, std=1e-3, dtype=torch.float32) * loud).square() * inside
    s = dict(case=case, step=100, seed=int(torch.randint(1 << 30, (1,), generator=d.g, device=DEV)), grad=g)
    s["p"] = p if case["param"] == "f32" else p.to(torch.bfloat16)
    if case["param"] == "master":
        s["master"] = p
    if case["state"] == "q8":
        s["m"], s["m_scale"] = _encode(m, None, signed=True)
        s["v"], s["v_scale"] = _encode(v.sqrt(), None, signed=False)
    else:
        s["m"], s["v"] = m, v
    if own:
        from bit_quantized_amd import block
        cut = lambda t: [t[a:a + n] for a, n in zip(at, sizes)]                      # noqa: E731
        s["op"] = block.AdamW(cut(s["p"]), cut(g), masters=cut(p) if case["param"] == "master" else None, state=case["state"],
                              seed=s["seed"], arena={k: s[k] for k in ("m", "v", "m_scale", "v_scale") if k in s}, **HYPER)
        s["op"].steps = s["step"]
    return s


# ------------------------------------------------------------------------------------------------- one pass
def run(state):
    return {"norm": _run_norm, "rope": _run_rope, "attn": _run_attn, "adamw": _run_adamw}[state["case"]["op"]](state)


def _heads(t, case, which):
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    lo, n = {"q": (0, hq), "k": (hq, hkv), "v": (hq + hkv, hkv)}[which]
    return t[:, lo * dim:(lo + n) * dim].unflatten(1, (n, dim))


def _normed(x, kind, eps=1e-6):
    """(x normalized along its last axis, the mean taken off, one over the deviation)"""
    mean = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[..., :1])
    rstd = torch.rsqrt((x - mean).square().mean(-1, keepdim=True) + eps)
    return (x - mean) * rstd, mean, rstd


def _normed_back(dn, n, rstd, kind):
    """The gradient of what was normalized to n, from that of n."""
    dx = dn - n * (dn * n).mean(-1, keepdim=True)
    return (dx - dn.mean(-1, keepdim=True) if kind == "layer" else dx) * rstd


def _by_sample(t, seg):
    """Sums over the rows of each sample."""
    c = torch.arange(t.shape[0], device=t.device)
    which = (c[None, :] >= seg[:-1, None]) & (c[None, :] < seg[1:, None])
    return which.to(t.dtype) @ t


def _run_norm(s):
    case, x, y, seg = s["case"], s["x"], s.get("y"), s["seg"]
    c = case["chan"]
    shift, scale, gate = s["mod"][:, :c], s["mod"][:, c:2 * c], s["mod"][:, 2 * c:]
    if own:
        o = s["op"]
        r, h, stats = o.forward(x, y=y, gate=gate if y is not None else None, scale=scale, shift=shift, segments=seg)
        out = dict(h=h, r=r)
        if case["train"]:
            g = o.backward(s["dh"], s["dr"], r, y, stats, gate=gate if y is not None else None, scale=scale, shift=shift,
                           segments=seg)
            out.update({k: v for k, v in g.items() if v is not None})
        return out
    row = torch.bucketize(torch.arange(x.shape[0], device=DEV, dtype=torch.int32), seg[1:], right=True)
    f, low = torch.float32, torch.bfloat16
    w = s["weight"].to(f) if "weight" in s else torch.ones(c, device=DEV)
    wp = s["post_weight"].to(f) if "post_weight" in s else torch.ones(c, device=DEV)
    shift, scale, gate = (t.to(f)[row] for t in (shift, scale, gate))
    r = x.to(f)
    if y is not None:
        ny, _, ry = _normed(y.to(f), case["post"]) if case["post"] != "none" else (y.to(f), None, None)
        r = (r + gate * (ny * wp)).to(x.dtype).to(f)
    n, _, rr = _normed(r, case["norm"])
    out = dict(h=(n * w * (1 + scale) + shift).to(low), r=r.to(x.dtype))
    if case["train"]:
        dh = s["dh"].to(f)
        dx = s["dr"].to(f) + _normed_back(dh * (1 + scale) * w, n, rr, case["norm"])
        out.update(dx=dx.to(x.dtype), dscale=_by_sample(dh * n * w, seg).to(low), dshift=_by_sample(dh, seg).to(low))
        if "weight" in s:
            out["dweight"] = (dh * n * (1 + scale)).sum(0).to(low)
        if y is not None:
            dny = dx * gate * wp
            out["dy"] = (_normed_back(dny, ny, ry, case["post"]) if case["post"] != "none" else dny).to(low)
            out["dgate"] = _by_sample(dx * ny * wp, seg).to(low)
            if "post_weight" in s:
                out["dpost_weight"] = (dx * gate * ny).sum(0).to(low)
    return out


def _angles(case, pos):
    """The rotation angle of every token and pair."""
    axes = _ints(case["axes"])
    pairs = sum(axes) // 2
    axis = torch.cat([torch.full((a // 2,), i, dtype=torch.long) for i, a in enumerate(axes)]).to(DEV)
    if case["ladder"] == "shared":
        power = torch.arange(pairs, dtype=torch.float64) / pairs
    else:
        power = torch.cat([torch.arange(a // 2, dtype=torch.float64) / (a // 2) for a in axes])
    freq = torch.exp(-power * math.log(10000.0)).to(DEV)
    return pos.to(torch.float32)[:, axis] * freq.to(torch.float32)


def _turn(x, cos, sin, layout):
    """Rotates the pairs of x [M, H, D] by the angles with this cosine and sine [M, pairs]."""
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., 0::2], x[..., 1::2]) if layout == "pairs" else x.chunk(2, -1)
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack((u, v), -1).flatten(-2) if layout == "pairs" else torch.cat((u, v), -1)


def _run_rope(s):
    case = s["case"]
    q, k = _heads(s["qkv"], case, "q"), _heads(s["qkv"], case, "k")
    if own:
        o = s["op"]
        q2, k2 = o.forward(q, k, s["pos"])
        if not case["train"]:
            return dict(q=q2, k=k2)
        g = o.backward(s["dq"], s["dk"], q, k, s["pos"])
        return dict(q=q2, k=k2, **{n: t for n, t in g.items() if t is not None})
    f, low = torch.float32, torch.bfloat16
    angle = _angles(case, s["pos"])
    cos, sin = angle.cos(), angle.sin()
    out = {}
    for n, x in (("q", q), ("k", k)):
        x = x.to(f)
        norm, _, rstd = _normed(x, "rms") if case["normed"] else (x, None, None)
        w = s["w" + n].to(f) if case["normed"] else 1.0
        out[n] = _turn(norm * w, cos, sin, case["layout"]).to(low)
        if case["train"]:
            dn = _turn(s["d" + n].to(f), cos, -sin, case["layout"])
            out["d" + n] = (_normed_back(dn * w, norm, rstd, "rms") if case["normed"] else dn).to(low)
            if case["normed"]:
                out["dw" + n] = (dn * norm).sum((0, 1)).to(low)
    return out


def _seen(n, prefix, mask):
    """Which key (last axis) each query of a document of n tokens sees."""
    i = torch.arange(n, device=DEV)
    return torch.ones(n, n, dtype=torch.bool, device=DEV) if mask == "full" else (i[None, :] <= i[:, None]) | (i[None, :] < prefix)


def _one_doc(q, k, v, do, seen, cap):
    """Attention of one document, heads first, keys and values already repeated: (o, lse, dq, dk, dv)."""
    c = q.shape[-1] ** -0.5
    s = (q @ k.transpose(1, 2).contiguous()) * c
    if cap:
        t = torch.tanh(s / cap)
        s = t * cap
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    lse, p = (top + total.log())[..., 0], p / total
    o = p @ v
    if do is None:
        return o, lse, None, None, None
    dp = do @ v.transpose(1, 2).contiguous()
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    if cap:
        ds = ds * (1 - t * t)
    ds = ds * c
    return o, lse, ds @ k, ds.transpose(1, 2).contiguous() @ q, p.transpose(1, 2).contiguous() @ do


def _plain_attn(s, f):
    """All documents, in the type f, unrounded."""
    case, first = s["case"], s["first"]
    hq, hkv, m = case["hq"], case["hkv"], s["q"].shape[0]
    v = _heads(s["qkv"], case, "v")
    o, dq = (torch.zeros(hq, m, case["dim"], device=DEV, dtype=f) for _ in range(2))
    dk, dv = (torch.zeros(hkv, m, case["dim"], device=DEV, dtype=f) for _ in range(2))
    lse = torch.full((hq, m), -math.inf, device=DEV, dtype=f)
    a = first
    for n, prefix in zip(_ints(case["docs"]), _prefixes(case)):
        at = slice(a, a + n)
        a += n
        if n:
            part = [None if t is None else t[at].to(f).transpose(0, 1).repeat_interleave(hq // t.shape[1], 0).contiguous()
                    for t in (s["q"], s["k"], v, s.get("do"))]
            o[:, at], lse[:, at], *g = _one_doc(*part, _seen(n, prefix, case["mask"]), case["cap"])
            if case["train"]:
                dq[:, at], dk[:, at], dv[:, at] = g[0], *(t.unflatten(0, (hkv, hq // hkv)).sum(1) for t in g[1:])
    return [t.transpose(0, 1) for t in (o, dq, dk, dv)] + [lse]


def _run_attn(s):
    case = s["case"]
    if own:
        q, k, v, op = s["q"], s["k"], _heads(s["qkv"], case, "v"), s["op"]
        o, lse = op.forward(q, k, v, docs=s["docs"], prefix=s["prefix"])
        if not case["train"]:
            return dict(o=o, lse=lse)
        dq, dk, dv = op.backward(s["do"], q, k, v, o, lse, docs=s["docs"], prefix=s["prefix"])
        return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)
    o, dq, dk, dv, lse = _plain_attn(s, torch.float32)
    low = torch.bfloat16
    out = dict(o=o.to(low), lse=lse)
    return dict(out, dq=dq.to(low), dk=dk.to(low), dv=dv.to(low)) if case["train"] else out


# An 8-bit state holds a block of 128 elements as codes times one 32-bit scale, the block's largest magnitude. A code is a
# number with 4 fraction bits whose largest, 1.9375 * 2^(top - 1), stands for the scale: signed, 3 exponent bits and a sign
# for the first moment; unsigned, 4 exponent bits for the root of the second.
_TOP = {True: 127, False: 255}


def _value(code):
    """What a code without sign stands for, in units of its smallest."""
    e = (code >> 4).to(torch.int32)
    frac = (code & 15).to(torch.float32)
    return torch.where(e > 0, torch.ldexp(frac + 16, (e - 1).clamp(min=0)), frac)


def _most(signed):
    return 31.0 * 2.0 ** ((_TOP[signed] >> 4) - 1)


def _decode(code, scale, signed):
    c = code.to(torch.int32)
    v = _value(c & _TOP[signed]) * (scale * (1 / _most(signed))).repeat_interleave(128)
    return torch.where(c > 127, -v, v) if signed else v


def _encode(x, bits, signed):
    """Codes and scales of x [n blocks of 128]: rounded down after `bits` / 2^19 of a code's step is added (None: a half)."""
    scale = x.view(-1, 128).abs().amax(1)
    unit = torch.where(scale > 1e-35, scale.reciprocal() * _most(signed), torch.zeros_like(scale))
    y = x.abs() * unit.repeat_interleave(128)
    y = torch.where(y < 16, (y + 16) - 16, y)                                         # 19 bits below a code's step, as above 16
    e = torch.frexp(y)[1].clamp(min=5) - 5                                            # the exponent of a code's step
    frac = torch.ldexp(y.to(torch.float64), -e) + (0.5 if bits is None else bits.to(torch.float64) * 2.0 ** -19)
    frac = frac.floor().to(torch.int64)                                               # 16 to 32, below 16 at the bottom
    code = (frac + 16 * e).clamp(max=_TOP[signed])
    code = torch.where((code == 0) & (x != 0), 1, code) if not signed else code      # a root above zero stays above it
    code = code + 128 * (x < 0) if signed else code
    return code.to(torch.uint8), scale


def _bits(n, seed, step):
    """32 random bits for each element: a mix of its place with the step's key (odd numbers from the golden ratio and from
    the roots of 2, 3 and 11)."""
    mask = 0xFFFFFFFF
    key = (seed * 0x9E3779B1 + step * 0x510E527F) & mask
    h = (torch.arange(n, device=DEV, dtype=torch.int64) * 0x9E3779B1 + key) & mask
    h = ((h ^ (h >> 16)) * 0x6A09E667) & mask
    h = ((h ^ (h >> 15)) * 0xBB67AE85) & mask
    return h ^ (h >> 16)


def _run_adamw(s):
    case = s["case"]
    if own:
        s["op"].step()
    else:
        s["step"] += 1
        _plain_adamw(s, torch.float32)
    out = dict(p=s["p"])
    if case["param"] == "master":
        out["master"] = s["master"]
    if case["state"] == "f32":
        return dict(out, m=s["m"], v=s["v"])
    return dict(out, m=_decode(s["m"], s["m_scale"], True), root_v=_decode(s["v"], s["v_scale"], False))


def _f32(x):
    """A host number rounded to 32 bits."""
    return torch.tensor(x, dtype=torch.float32).item()


def _plain_adamw(s, f):
    case, t = s["case"], s["step"]
    b1, b2 = HYPER["betas"]
    decay, rate = _f32(1 - HYPER["lr"] * HYPER["weight_decay"]), _f32(HYPER["lr"] / (1 - b1 ** t))
    lift = _f32(1 / math.sqrt(1 - b2 ** t))
    p, g = s.get("master", s["p"]).to(f), s["grad"].to(f)
    if case["state"] == "q8":
        m, v = _decode(s["m"], s["m_scale"], True), _decode(s["v"], s["v_scale"], False).square()
    else:
        m, v = s["m"], s["v"]
    m = m * _f32(b1) + g * _f32(1 - b1)
    v = v * _f32(b2) + (g * g) * _f32(1 - b2)
    root = v.sqrt()
    p = p * decay - (m / (root * lift + HYPER["eps"])) * rate
    bits = _bits(p.numel(), s["seed"], t) if case["state"] == "q8" or case["param"] == "bf16" else None
    if case["state"] == "q8":
        new = _encode(m, bits >> 13, True), _encode(root, ((bits * 0x9E3779B1) & 0xFFFFFFFF) >> 13, False)
        for (code, scale), n in zip(new, "mv"):
            s[n].copy_(code)
            s[n + "_scale"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    if case["param"] == "bf16":                                                       # no master: rounded at random
        u = p.view(torch.int32) + (((bits * 0x510E527F) & 0xFFFFFFFF) >> 16).to(torch.int32)
        s["p"].copy_((u & -65536).view(torch.float32))
    elif case["param"] == "master":
        s["master"].copy_(p)
        s["p"].copy_(p)
    else:
        s["p"].copy_(p)


# ------------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """What run() returns, from the definitions, in 64 bits."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"norm": _exact_norm, "rope": _exact_rope, "attn": _exact_attn, "adamw": _exact_adamw}[case["op"]](s)


def _exact_norm(s):
    case, seg = s["case"], s["seg"].tolist()
    c, d = case["chan"], torch.float64
    mod = s["mod"].to(d)
    w = s["weight"].to(d) if "weight" in s else torch.ones(c, dtype=d, device=DEV)
    wp = s["post_weight"].to(d) if "post_weight" in s else torch.ones(c, dtype=d, device=DEV)
    x = s["x"].to(d).requires_grad_(True)
    y = s["y"].to(d).requires_grad_(True) if "y" in s else None
    mod.requires_grad_(True), w.requires_grad_(True), wp.requires_grad_(True)

    def norm(t, kind):
        if kind == "layer":
            t = t - t.mean(1, keepdim=True)
        return t / torch.sqrt((t * t).mean(1, keepdim=True) + 1e-6)

    rs, hs = [], []
    for b in range(len(seg) - 1):
        at = slice(seg[b], seg[b + 1])
        shift, scale, gate = mod[b, :c], mod[b, c:2 * c], mod[b, 2 * c:]
        r = x[at]
        if y is not None:
            r = r + gate * (wp * (norm(y[at], case["post"]) if case["post"] != "none" else y[at]))
            r = r + (r.detach().to(s["x"].dtype).to(d) - r.detach())                 # the stream is held in its type
        rs.append(r)
        hs.append((1 + scale) * (w * norm(r, case["norm"])) + shift)
    r, h = torch.cat(rs), torch.cat(hs)
    out = dict(h=h.detach(), r=r.detach())
    if case["train"]:
        wanted = dict(dx=x, mod=mod)
        wanted.update(dict(dy=y) if y is not None else {})
        wanted.update(dict(dweight=w) if "weight" in s else {})
        wanted.update(dict(dpost_weight=wp) if "post_weight" in s else {})
        total = (h * s["dh"].to(d)).sum() + (r * s["dr"].to(d)).sum()
        got = dict(zip(wanted, torch.autograd.grad(total, list(wanted.values()))))
        dm = got.pop("mod")
        out.update(got, dshift=dm[:, :c], dscale=dm[:, c:2 * c])
        if y is not None:
            out["dgate"] = dm[:, 2 * c:]
    return out


def _exact_rope(s):
    case, d = s["case"], torch.float64
    dim, layout = case["dim"], case["layout"]
    axes = _ints(case["axes"])
    half = dim // 2
    pairs = [(2 * j, 2 * j + 1) if layout == "pairs" else (j, j + half) for j in range(half)]
    owner = [(i, j / (a // 2)) for i, a in enumerate(axes) for j in range(a // 2)]
    turn = torch.zeros(s["pos"].shape[0], half, dtype=torch.complex128, device=DEV)
    for j, (axis, power) in enumerate(owner):
        power = j / half if case["ladder"] == "shared" else power
        turn[:, j] = torch.polar(torch.ones_like(s["pos"][:, axis], dtype=d), s["pos"][:, axis].to(d) * 10000.0 ** -power)
    a, b = (torch.tensor(t, device=DEV) for t in zip(*pairs))
    out = {}
    for n in "qk":
        x = _heads(s["qkv"], case, n).to(d).requires_grad_(True)
        w = s["w" + n].to(d).requires_grad_(True) if case["normed"] else None
        t = x * w / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) if case["normed"] else x
        z = torch.complex(t[..., a], t[..., b]) * turn[:, None]
        y = torch.zeros_like(x).index_copy(-1, a, z.real).index_copy(-1, b, z.imag)
        out[n] = y.detach()
        if case["train"]:
            g = torch.autograd.grad((y * s["d" + n].to(d)).sum(), [x] + ([w] if case["normed"] else []))
            out["d" + n] = g[0]
            if case["normed"]:
                out["dw" + n] = g[1]
    return out


def _exact_attn(s):
    case, d = s["case"], torch.float64
    hq, hkv, dim, m = case["hq"], case["hkv"], case["dim"], s["q"].shape[0]
    q, k, v = s["q"], s["k"], s["qkv"][:, (hq + hkv) * dim:].reshape(m, hkv, dim)
    o, dq = (torch.zeros(m, hq, dim, dtype=d, device=DEV) for _ in range(2))
    dk, dv = (torch.zeros(m, hkv, dim, dtype=d, device=DEV) for _ in range(2))
    lse = torch.full((hq, m), -math.inf, dtype=d, device=DEV)
    start = s["docs"].tolist()
    for b, (lo, hi) in enumerate(zip(start, start[1:])):
        if hi == lo:
            continue
        i = torch.arange(hi - lo, device=DEV)
        hidden = torch.zeros(hi - lo, hi - lo, dtype=torch.bool, device=DEV)
        if case["mask"] != "full":
            hidden = (i[None] > i[:, None]) & (i[None] >= int(s["prefix"][b]))
        for h in range(hq):
            g = h * hkv // hq
            a, e, u = (t[lo:hi, j].to(d) for t, j in ((q, h), (k, g), (v, g)))
            z = a @ e.T / math.sqrt(dim)
            slope = 1.0
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
                slope = 1 - (z / case["cap"]).square()
            z = z.masked_fill(hidden, -math.inf)
            lse[h, lo:hi] = torch.logsumexp(z, 1)
            p = torch.exp(z - lse[h, lo:hi, None])
            o[lo:hi, h] = p @ u
            if case["train"]:
                grad = s["do"][lo:hi, h].to(d)
                dz = p * (grad @ u.T - (grad * o[lo:hi, h]).sum(1, keepdim=True)) * slope / math.sqrt(dim)
                dq[lo:hi, h] = dz @ e
                dk[lo:hi, g] += dz.T @ a
                dv[lo:hi, g] += p.T @ grad
    out = dict(o=o, lse=lse)
    return dict(out, dq=dq, dk=dk, dv=dv) if case["train"] else out


def _exact_adamw(s):
    case, d, t = s["case"], torch.float64, s["step"] + 1
    (b1, b2), lr = HYPER["betas"], HYPER["lr"]
    g = s["grad"].to(d)

    def of_codes(code, scale, signed):
        e, frac = torch.div(code.to(d) % (128 if signed else 256), 16, rounding_mode="floor"), code.to(d) % 16
        val = torch.where(e > 0, (16 + frac) * 2 ** (e - 1), frac) / (31 * 64 if signed else 31 * 2 ** 14)
        val = (val.view(-1, 128) * scale.to(d)[:, None]).view(-1)
        return torch.where(code > 127, -val, val) if signed else val

    def to_value(x, bits, signed):
        """x in the 8-bit form, as the value that it stands for."""
        most, top = (31 * 64, 127) if signed else (31 * 2 ** 14, 255)
        big = x.abs().view(-1, 128).amax(1, keepdim=True).expand(-1, 128).reshape(-1)
        y = torch.where(big > 1e-35, x.abs() * most / big, torch.zeros_like(x))
        step = 2.0 ** (torch.floor(torch.log2(y.clamp(min=16.0))) - 4)
        y = (torch.floor(y / step + bits.to(d) / 2 ** 19) * step).clamp(max=most)
        y = torch.where((y == 0) & (x != 0), 1.0, y) if not signed else y
        return torch.sign(x) * y * big / most

    if case["state"] == "q8":
        m, v = of_codes(s["m"], s["m_scale"], True), of_codes(s["v"], s["v_scale"], False).square()
    else:
        m, v = s["m"].to(d), s["v"].to(d)
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    p = s.get("master", s["p"]).to(d)
    p = p - lr * HYPER["weight_decay"] * p - lr * (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + HYPER["eps"])
    bits = _bits(p.numel(), s["seed"], t)
    out = dict(p=p)
    if case["param"] == "bf16":
        step = 2.0 ** (torch.frexp(p)[1] - 8).to(d)
        out["p"] = torch.sign(p) * torch.floor(p.abs() / step + (((bits * 0x510E527F) & 0xFFFFFFFF) >> 16).to(d) / 65536) * step
    if case["param"] == "master":
        out["master"] = p
    if case["state"] == "f32":
        return dict(out, m=m, v=v)
    return dict(out, m=to_value(m, bits >> 13, True), root_v=to_value(v.sqrt(), ((bits * 0x9E3779B1) & 0xFFFFFFFF) >> 13, False))
