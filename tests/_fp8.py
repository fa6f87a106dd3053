"""Plain 64-bit definitions of the FP8 and routing operators, in numpy."""
from __future__ import annotations

import numpy as np
import torch

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _table():
    """The value of each e4m3 byte: sign, four exponent bits (bias 7), three of the fraction; 0x7F is NaN."""
    v = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        x = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v[b] = (np.nan if b & 0x7F == 0x7F else x) * (-1 if b & 0x80 else 1)
    return v


E4M3 = _table()
POSITIVE = E4M3[:0x7F]  # ascending


def encode(x):
    """The nearest e4m3 value (half to even) of each number, as a float; NaN stays NaN."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(POSITIVE, a), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    up, down = POSITIVE[hi] - a, a - POSITIVE[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)) | (up == 0), hi, lo)
    return np.where(np.isnan(x), np.nan, np.copysign(POSITIVE[pick], x))


def bytes_of(t):
    """A float8 tensor's values, by the table."""
    return E4M3[t.contiguous().view(torch.uint8).cpu().numpy()]


def quantize(x, tall=1):
    """(values, scales) of float32 x with a scale for each tall x 128 block; the quotients are rounded to FP32."""
    n, k = x.shape
    nb, kb = -(-n // tall), -(-k // 128)
    q, s = np.empty((n, k)), np.empty((nb, kb), np.float32)
    for i in range(nb):
        for b in range(kb):
            blk = x[i * tall:(i + 1) * tall, b * 128:(b + 1) * 128].astype(np.float64)
            most = np.abs(blk).max() if np.isfinite(blk).all() else np.nan
            s[i, b] = np.float32(max(most, 2.0 ** -64) / 448.0) if most == most else np.nan
            with np.errstate(invalid="ignore"):
                q[i * tall:(i + 1) * tall, b * 128:(b + 1) * 128] = encode((blk / np.float64(s[i, b])).astype(np.float32))
    return q, s


def values(q, s, tall=1):
    """What e4m3 values (numpy) with scales stand for."""
    n, k = q.shape
    return q * s.astype(np.float64)[np.arange(n) // tall][:, np.arange(k) // 128]


def random_bytes(rows, cols, seed, pad=0, offset=0, whole=False):
    """An e4m3 GPU matrix of random finite bytes with row stride cols + pad, its first byte `offset` past a 16-byte
    boundary; what lies outside it is NaN. whole: small integers only."""
    g = torch.Generator().manual_seed(seed)
    if whole:
        b = torch.randint(-4, 5, (rows, cols), generator=g).float().to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        b = torch.randint(0, 0x77, (rows, cols), generator=g, dtype=torch.uint8)
        b |= torch.randint(0, 2, (rows, cols), generator=g, dtype=torch.uint8) << 7
    ld = cols + pad
    room = torch.full((offset + rows * ld + 64,), 0x7F, dtype=torch.uint8)
    room[offset:offset + rows * ld].view(rows, ld)[:, :cols] = b
    room = room.to("cuda")
    return room[offset:offset + rows * ld].view(torch.float8_e4m3fn).view(rows, ld)[:, :cols]


def random_scales(rows, blocks, seed, by_block=True, powers=False):
    g = torch.Generator().manual_seed(seed + 1000)
    s = torch.exp2(torch.randint(-3, 4, (rows, blocks), generator=g).float()) if powers else \
        torch.rand(rows, blocks, generator=g) * 0.1 + 1e-3
    return s.t().contiguous().to("cuda").t() if by_block else s.to("cuda")


def half_step(kind):
    """Half a step of the type, relative to the value, and half its least step."""
    return {"fp32": (2.0 ** -24, 2.0 ** -150), "bf16": (2.0 ** -8, 2.0 ** -134), "fp16": (2.0 ** -11, 2.0 ** -25)}[kind]


def product_bound(want, magnitude, K, kind):
    """The error a product's element may have: a block's 128 additions in the matrix unit, each off by a whole FP32
    step at most; then for each block the two scales' product and one fused multiply-add; then the rounding to C. With
    a 16-bit C the FP8 matrix unit drops of seven products in a group of eight less than 2^-13 of the largest each."""
    rel, least = half_step(kind)
    blocks = -(-K // 128)
    inside = (128 * 2.0 ** -23 + (blocks + 1) * 2.0 ** -24 + (0.0 if kind == "fp32" else 7 * 2.0 ** -13)) * magnitude
    return inside + rel * (np.abs(want) + inside) + least


def route(logits, k, bias=None, score="softmax", groups=1, top_groups=1, renorm=True, scale=1.0):
    """(weights, ids, scores) in 64 bits, a token at a time."""
    T, E = logits.shape
    W, I, S = np.zeros((T, k)), np.zeros((T, k), np.int64), np.zeros((T, E))
    for t in range(T):
        l = logits[t].astype(np.float64)
        with np.errstate(over="ignore", invalid="ignore"):
            s = np.exp(l - l.max()) if score == "softmax" else 1 / (1 + np.exp(-l))
            s = s / s.sum() if score == "softmax" else s
            c = s if bias is None else s + bias.astype(np.float64)
        c = np.where(np.isnan(c), -np.inf, c)
        able = np.ones(E, bool)
        if groups > 1:
            by = c.reshape(groups, -1)
            strength = -np.sort(-by, 1)[:, :2].sum(1)
            able = np.isin(np.arange(E) // (E // groups), np.lexsort((np.arange(groups), -strength))[:top_groups])
        at = np.arange(E)[able]
        ids = at[np.lexsort((at, -c[able]))][:k]
        total = s[ids].sum() if renorm else 1.0
        W[t], I[t], S[t] = scale * s[ids] / total if total else 0.0, ids, s
    return W, I, S


def route_grad(S, I, dW, score, renorm, scale):
    """The gradient of the logits by the chain rule, a token at a time, from the Jacobian of the weights."""
    T, E = S.shape
    out = np.zeros((T, E))
    for t in range(T):
        s, ids = S[t], I[t]
        k = len(ids)
        jac = np.eye(E) * s - np.outer(s, s) if score == "softmax" else np.diag(s * (1 - s))  # ds_a/dl_b
        total = s[ids].sum()
        by_s = scale * (np.eye(k) / total - s[ids][:, None] / total ** 2) if renorm else scale * np.eye(k)
        out[t] = dW[t] @ by_s @ jac[ids]
    return out


def plan(ids, experts):
    flat = np.where((ids < 0) | (ids >= experts), experts, ids).reshape(-1)
    order = np.argsort(flat, kind="stable")
    place = np.empty_like(order)
    place[order] = np.arange(len(order))
    return np.searchsorted(flat[order], np.arange(experts + 1)), order // ids.shape[1], place.reshape(ids.shape)
