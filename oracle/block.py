"""Plain float64 implementations of what the library computes around the
linears: the gated residual and modulated norm, the rotation by positions on
several axes, attention inside packed documents, and the AdamW step, each
with its gradient by the formulas.  Test infrastructure: it shares no code
with the library and is slow on purpose.
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------ norm
def norm_rows(x, kind, eps):
    """(n, mean, rstd) of rows x [M, C]; kind "rms", "layer" or "none"."""
    if kind == "none":
        return x, np.zeros((len(x), 1)), np.ones((len(x), 1))
    mean = x.mean(1, keepdims=True) if kind == "layer" else np.zeros((len(x), 1))
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    return (x - mean) * rstd, mean, rstd


def norm_grad(dn, n, rstd, kind):
    """Gradient of the rows that were normalized to n."""
    if kind == "none":
        return dn
    t = dn - n * (dn * n).mean(1, keepdims=True)
    if kind == "layer":
        t = t - dn.mean(1, keepdims=True)
    return rstd * t


def samples_of(offsets, M):
    """The sample of each row: the last one that starts at or before it."""
    starts = np.asarray(offsets[:-1])
    return np.array([max([b for b in range(len(starts)) if starts[b] <= i], default=0) for i in range(M)], dtype=int)


def gated_residual(x, y, which, gate, post_weight, post_norm, eps, alpha):
    """r = x + alpha gate_b (post_weight N_post(y)), unrounded."""
    n, _, _ = norm_rows(y, post_norm, eps)
    return x + alpha * gate[which] * (post_weight * n)


def modulated_norm(r, which, scale, shift, weight, norm, eps):
    """h = (1 + scale_b) (weight N(r)) + shift_b"""
    n, _, _ = norm_rows(r, norm, eps)
    return (1 + scale[which]) * (weight * n) + shift[which]


def norm_backward(dh, dr, r, y, which, n_seg, gate, scale, weight, post_weight, norm, post_norm, eps, alpha):
    """Gradients by name, and under the same name with "|" before it the sum
    of the magnitudes of the terms each one adds up."""
    g = {}
    dx, mag = dr.copy(), np.abs(dr)
    by = lambda t: np.stack([t[which == b].sum(0) for b in range(n_seg)])
    if dh is not None:
        n, _, rstd = norm_rows(r, norm, eps)
        a = dh * (1 + scale[which]) * weight
        dx = dx + norm_grad(a, n, rstd, norm)
        mag = mag + rstd * (np.abs(a) + np.abs(n) * np.abs(a * n).mean(1, keepdims=True)
                            + np.abs(a).mean(1, keepdims=True))
        g["dscale"], g["|dscale"] = by(dh * n * weight), by(np.abs(dh * n * weight))
        g["dshift"], g["|dshift"] = by(dh), by(np.abs(dh))
        t = dh * n * (1 + scale[which])
        g["dweight"], g["|dweight"] = t.sum(0), np.abs(t).sum(0)
    g["dx"], g["|dx"] = dx, mag
    if y is not None:
        m, _, ry = norm_rows(y, post_norm, eps)
        e = alpha * dx * gate[which] * post_weight
        g["dy"] = norm_grad(e, m, ry, post_norm)
        f = np.abs(alpha * mag * gate[which] * post_weight)
        g["|dy"] = ry * (f + np.abs(m) * (f * np.abs(m)).mean(1, keepdims=True) + f.mean(1, keepdims=True))
        g["dgate"], g["|dgate"] = by(alpha * dx * post_weight * m), by(np.abs(alpha * mag * post_weight * m))
        t = alpha * dx * gate[which] * m
        g["dpost_weight"], g["|dpost_weight"] = t.sum(0), np.abs(alpha * mag * gate[which] * m).sum(0)
    return g


# ------------------------------------------------------------------ rope
def rope_angles(positions, axis_dims, theta, ladder):
    """Angle of every row and pair."""
    cols = []
    pairs = sum(axis_dims) // 2
    for axis, dims in enumerate(axis_dims):
        for i in range(dims // 2):
            power = len(cols) / pairs if ladder == "shared" else 2 * i / dims
            cols.append(positions[:, axis].astype(np.float64) * theta ** -power)
    return np.stack(cols, 1)


def rope_turn(t, angle, layout):
    """Rotate the pairs of t [M, H, D]."""
    out = t.copy()
    pairs = angle.shape[1]
    for j in range(pairs):
        a, b = (2 * j, 2 * j + 1) if layout == "pairs" else (j, j + pairs)
        c, s = np.cos(angle[:, j])[:, None], np.sin(angle[:, j])[:, None]
        out[:, :, a] = t[:, :, a] * c - t[:, :, b] * s
        out[:, :, b] = t[:, :, a] * s + t[:, :, b] * c
    return out


def rope_forward(x, angle, layout, weight, eps):
    if weight is not None:
        x = weight * x / np.sqrt((x * x).mean(2, keepdims=True) + eps)
    return rope_turn(x, angle, layout)


def rope_backward(d, x, angle, layout, weight, eps):
    """(gradient of x, of the weight)"""
    u = rope_turn(d, -angle, layout)
    if weight is None:
        return u, None
    rstd = 1 / np.sqrt((x * x).mean(2, keepdims=True) + eps)
    n = x * rstd
    t = u * weight
    return rstd * (t - n * (t * n).mean(2, keepdims=True)), (u * n).sum((0, 1))


# ------------------------------------------------------------------ attention
def visible(n, mask, prefix):
    """Which keys (columns) the queries (rows) of a document of n rows see."""
    i = np.arange(n)
    if mask == "full":
        return np.ones((n, n), dtype=bool)
    return (i[None, :] <= i[:, None]) | ((i[None, :] < prefix) if mask == "prefix" else False)


def attention_head(q, k, v, see, scale, cap):
    """(o, lse, p, slope) of one document and head."""
    s = scale * (q @ k.T)
    slope = np.ones_like(s)
    if cap:
        t = np.tanh(s / cap)
        s, slope = cap * t, 1 - t * t
    s = np.where(see, s, -np.inf)
    top = s.max(1, keepdims=True)
    p = np.exp(s - top)
    total = p.sum(1, keepdims=True)
    p = p / total
    return p @ v, (top + np.log(total))[:, 0], p, slope


def attention_head_grad(q, k, v, do, o, p, slope, scale):
    """(dq, dk, dv, ds): ds is the gradient of scale-free scores, dP weighted."""
    dp = do @ v.T
    ds = p * (dp - (do * o).sum(1, keepdims=True)) * slope
    return scale * ds @ k, scale * ds.T @ q, p.T @ do, ds


# ------------------------------------------------------------------ AdamW
def adamw(p, g, m, v, t, lr, b1, b2, eps, wd):
    """(p, m, v) after step t."""
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    return p - lr * wd * p - lr * (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps), m, v


def code_values(signed):
    """What each of the 256 codes of an 8-bit state stands for, in units of the largest."""
    bits = 7 if signed else 8
    vals = np.array([(c % 16) if c < 16 else (16 + c % 16) * 2.0 ** (c // 16 - 1) for c in range(1 << bits)])
    vals = vals / vals[-1]
    return np.concatenate([vals, -vals]) if signed else vals


def code_round(x, scale, bits, signed):
    """Codes of the magnitudes in x for a block scale, rounded down after bits / 2^19
    of a step is added; one block."""
    vals = code_values(signed)[:128 if signed else 256]
    codes = np.zeros(x.shape, dtype=np.int64)
    for i, a in enumerate(np.abs(x) / scale if scale > 0 else np.zeros(x.shape)):
        a *= 1 + 2.0 ** -50             # (the quotient's own rounding must not fall below a code)
        c = int(np.searchsorted(vals, a, side="right") - 1)
        if c + 1 < len(vals):
            frac = (a - vals[c]) / (vals[c + 1] - vals[c])
            c += int(frac + bits[i] / 2.0 ** 19 >= 1)
        if not signed and c == 0 and x[i] != 0:
            c = 1
        codes[i] = c + (128 if signed and x[i] < 0 else 0)
    return codes


def mixed_bits(i, seed, t):
    """The 32 random bits of arena place i at step t."""
    mask = (1 << 32) - 1
    h = (int(i) * 0x9E3779B1 + seed * 0x9E3779B1 + t * 0x510E527F) & mask
    h = ((h ^ (h >> 16)) * 0x6A09E667) & mask
    h = ((h ^ (h >> 15)) * 0xBB67AE85) & mask
    return h ^ (h >> 16)


def half_step(v, mantissa):
    """Half the spacing of a float type with that many mantissa bits at |v|."""
    return np.ldexp(1.0, np.frexp(np.maximum(np.abs(v), 1e-38))[1] - mantissa - 1)

