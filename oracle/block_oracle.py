"""float64 oracle of the operators around the layer: residual addition with the
root-mean-square norm (forward, backward, 8-bit output), dropout, 4-bit weights
and the SwiGLU experts on them.  numpy only; test infrastructure, like the other
oracles here, and written from the definitions in include/moe.h.

Values are float64 arrays that hold what the device tensors hold; `rounder`
arguments round to a storage type (identity by default)."""
from __future__ import annotations

import numpy as np


def philox4x32_10(counter, key):
    """Philox4x32 with ten rounds (Salmon et al., "Parallel Random Numbers: As
    Easy as 1, 2, 3", SC 2011): counter [..., 4] uint32 values, key (k0, k1)."""
    c = [np.asarray(counter[..., i], dtype=np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    mask = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        hi0, lo0 = np.divmod(c[0] * np.uint64(0xD2511F53), np.uint64(1 << 32))
        hi1, lo1 = np.divmod(c[2] * np.uint64(0xCD9E8D57), np.uint64(1 << 32))
        c = [(hi1 ^ c[1] ^ np.uint64(k[0])) & mask, lo1, (hi0 ^ c[3] ^ np.uint64(k[1])) & mask, lo0]
        k = [(k[0] + 0x9E3779B9) % (1 << 32), (k[1] + 0xBB67AE85) % (1 << 32)]
    return np.stack(c, -1)


def keep_mask(rows, cols, p, seed, offset):
    """True where the dropout keeps an element, one element at a time."""
    thr = int(np.floor(p * 65536 + 0.5))
    nb = (cols + 7) // 8
    ctr = np.zeros((rows, nb, 4), dtype=np.uint64)
    ctr[..., 0] = np.arange(nb)[None, :]
    ctr[..., 1] = np.arange(rows)[:, None]
    ctr[..., 2] = offset % (1 << 32)
    ctr[..., 3] = offset >> 32
    w = philox4x32_10(ctr, (seed % (1 << 32), seed >> 32))
    mask = np.zeros((rows, cols), dtype=bool)
    for c in range(cols):
        word = w[:, c // 8, (c % 8) // 2]
        number = word >> np.uint64(16) if c % 2 else word % np.uint64(65536)
        mask[:, c] = number >= thr
    return mask


def dropout(x, p, seed, offset):
    thr = int(np.floor(p * 65536 + 0.5))
    if thr == 0:
        return x.copy()
    keep = keep_mask(*x.shape, p, seed, offset)
    out = np.zeros_like(x)
    if thr < 65536:
        out[keep] = x[keep] * (65536 / (65536 - thr))
    return out


def add_norm(x, residual, weight, eps, p=0.0, seed=0, offset=0, rounder=lambda v: v):
    """(h, y, rstd): h is rounded by `rounder` (the stream's type) before its norm."""
    h = dropout(x, p, seed, offset)
    if residual is not None:
        h = h + residual
    h = rounder(h)
    rstd = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    return h, h * rstd[:, None] * weight, rstd


def add_norm_bwd(dy, h, rstd, weight, dres=None, p=0.0, seed=0, offset=0):
    """(dh, dx, dw) from the saved h and rstd."""
    r = rstd[:, None]
    g = dy * weight
    dh = r * g - h * r ** 3 * (g * h).mean(-1, keepdims=True)
    if dres is not None:
        dh = dh + dres
    return dh, dropout(dh, p, seed, offset), (dy * h * r).sum(0)


def add_layer_norm(x, residual, weight, bias, eps, p=0.0, seed=0, offset=0, rounder=lambda v: v):
    """(h, y, mean, rstd): h is rounded by `rounder` (the stream's type) before its norm."""
    h = dropout(x, p, seed, offset)
    if residual is not None:
        h = h + residual
    h = rounder(h)
    mean = h.mean(-1)
    c = h - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(-1) + eps)
    y = c * rstd[:, None] * weight
    return h, y if bias is None else y + bias, mean, rstd


def add_layer_norm_bwd(dy, h, mean, rstd, weight, dres=None, p=0.0, seed=0, offset=0):
    """(dh, dx, dw, db) from the saved h, mean and rstd."""
    r = rstd[:, None]
    n = (h - mean[:, None]) * r
    g = dy * weight
    dh = r * (g - g.mean(-1, keepdims=True) - n * (g * n).mean(-1, keepdims=True))
    if dres is not None:
        dh = dh + dres
    return dh, dropout(dh, p, seed, offset), (dy * n).sum(0), dy.sum(0)


def numbers16(count, high, seed, offset):
    """The 16-bit numbers of `count` neighbouring places, counters (place / 8, high, offset)."""
    nb = (count + 7) // 8
    ctr = np.zeros((nb, 4), dtype=np.uint64)
    ctr[:, 0] = np.arange(nb)
    ctr[:, 1] = high
    ctr[:, 2] = offset % (1 << 32)
    ctr[:, 3] = offset >> 32
    w = philox4x32_10(ctr, (seed % (1 << 32), seed >> 32))
    r = np.zeros((nb, 8), dtype=np.int64)
    for j in range(8):
        r[:, j] = w[:, j // 2] >> np.uint64(16) if j % 2 else w[:, j // 2] % np.uint64(65536)
    return r.reshape(-1)[:count]


def e4m3_values(codes):
    """E4M3 codes (uint8) to the numbers that they stand for."""
    c = np.asarray(codes).astype(np.int64)
    e, f = c >> 3 & 15, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * np.exp2(e - 10.0))
    v = np.where((e == 15) & (f == 7), np.nan, v)
    return np.where(c & 128, -v, v)


def adamw_constants(lr, beta1, beta2, weight_decay, step):
    """(1 - b1, 1 - b2, 1 / sqrt(1 - b2^t), 1 - lr wd, lr / (1 - b1^t))"""
    return 1 - beta1, 1 - beta2, 1 / np.sqrt(1 - beta2 ** step), 1 - lr * weight_decay, lr / (1 - beta1 ** step)


def adamw(w, g, m, v, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, grad_scale=1.0, dtype=np.float64):
    """(w, m, v, root), each operation in `dtype`: with float32 what the device computes,
    operation by operation."""
    c = [dtype(x) for x in adamw_constants(lr, beta1, beta2, weight_decay, step)]
    w, g, m, v = (np.asarray(x, dtype=dtype) for x in (w, g, m, v))
    g = g * dtype(grad_scale)
    m = m * dtype(beta1) + g * c[0]
    v = v * dtype(beta2) + (g * g) * c[1]
    root = np.sqrt(v)
    return w * c[3] - m / (root * c[2] + dtype(eps)) * c[4], m, v, root


def state8(x, numbers, least):
    """float32 values to (codes' values, scales) of 128 each, rounded by `numbers`."""
    x = np.asarray(x, dtype=np.float32)
    n, one = len(x), np.float32(448)
    out, scales = np.zeros(n, dtype=np.float32), np.zeros((n + 127) // 128, dtype=np.float32)
    for b in range(len(scales)):
        at = slice(128 * b, min(n, 128 * b + 128))
        v = x[at]
        finite = np.isfinite(v)
        top = np.abs(v[finite]).max(initial=np.float32(0))
        inv = one * (np.float32(1) / top) if top >= np.float32(2.0 ** -100) else np.float32(0)
        z = np.minimum(np.abs(np.where(finite, v, np.float32(0))) * inv, one)
        step = np.exp2(np.floor(np.log2(np.maximum(z, 2.0 ** -6).astype(np.float64))) - 3)
        low = np.floor(z / step)
        q = (low + (z / step - low >= 1 - numbers[at] / 65536)) * step
        if least:
            q = np.where((z > 0) & (q == 0), 2.0 ** -9, q)
        out[at] = np.where(finite, np.copysign(q, v), np.nan)
        scales[b] = top * np.float32(1 / 448) if top >= np.float32(2.0 ** -100) else 0
    return out, scales


def w4_quantize(w, group, rounder):
    """codes [rows, K] 0..15 and scales [rows, K / group] (rounded by `rounder`)."""
    b = w.reshape(w.shape[0], -1, group)
    s = rounder(np.abs(b).max(-1) / 7)
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(s[..., None] > 0, b / s[..., None], 0.0)
    return (np.clip(np.rint(z), -8, 7) + 8).astype(np.uint8).reshape(w.shape), s


def w4_pack(codes):
    return (codes[..., 0::2] + 16 * codes[..., 1::2]).astype(np.uint8)


def w4_values(codes, scales):
    g = codes.shape[-1] // scales.shape[-1]
    return (codes.astype(np.float64) - 8) * np.repeat(scales, g, axis=-1)


def experts(x, topk_idx, gates, w_gate, w_up, w_down):
    """SwiGLU experts route by route; indices outside [0, E) add nothing."""
    out = np.zeros_like(x)
    E = w_gate.shape[0]
    for t in range(x.shape[0]):
        for j in range(topk_idx.shape[1]):
            e = int(topk_idx[t, j])
            if 0 <= e < E:
                h, u = w_gate[e] @ x[t], w_up[e] @ x[t]
                out[t] += gates[t, j] * (w_down[e] @ (h / (1 + np.exp(-h)) * u))
    return out
