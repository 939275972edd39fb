"""The prompt attention and the drafted trees' masks by their definitions in 64 bits, inputs of
the formats, and how far a result may be off, derived from the arithmetic that
include/mla_cache.h states."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

NOPE, ROPE, V = 128, 64, 128
SCALE = (NOPE + ROPE) ** -0.5
FP8 = (torch.float8_e4m3fn, torch.float8_e5m2)
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative


def values(shape, dtype, seed, mul=1.0):
    """Normal values in a format, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * mul
    if dtype in FP8:
        x = x.clamp(-448, 448)
    return x.to(dtype)


def f64(t):
    return t.float().double().numpy()


@dataclass
class Result:
    out: np.ndarray   # [T, H, 128]; tokens of no sequence NaN in all
    lse: np.ndarray   # [T, H]
    mag: np.ndarray   # [T, H, 128]: sum of weight * |v| / sum of weights
    flat: np.ndarray  # [T, H, 128]: sum of |v| / sum of weights (the largest weight is 1)
    dot: np.ndarray   # [T, H]: largest |scale| * sum |q k|
    reach: np.ndarray  # [T, H]: largest |scale| * max |q| * sum |k|
    longest: int


def attend(q, key, v, cu_q, cu_kv, scale, causal, limit=None):
    """q [T, H, 192], key [K, G, 192], v [K, G, 128] in float64; limit: the rows that exist."""
    T, H, _ = q.shape
    K, G = key.shape[0], key.shape[1]
    limit = K if limit is None else limit
    r = Result(*(np.full(s, np.nan) for s in ((T, H, V), (T, H), (T, H, V), (T, H, V), (T, H),
                                              (T, H))), 1)
    for s in range(len(cu_q) - 1):
        a, b = cu_q[s], min(cu_q[s + 1], T)
        n, m = cu_q[s + 1] - cu_q[s], cu_kv[s + 1] - cu_kv[s]
        last = max(0, min(cu_kv[s + 1], limit) - cu_kv[s]) if cu_kv[s] >= 0 else 0
        for t in range(a, b):
            seen = min(max(0, m - n + 1 + t - a if causal else m), last)
            for x in (r.out, r.mag, r.flat, r.dot, r.reach):
                x[t] = 0.0
            r.lse[t] = -np.inf
            if seen == 0:
                continue
            r.longest = max(r.longest, seen)
            kk = np.repeat(key[cu_kv[s]:cu_kv[s] + seen], H // G, 1)
            vv = np.repeat(v[cu_kv[s]:cu_kv[s] + seen], H // G, 1)
            x = scale * np.einsum("he,khe->hk", q[t], kk)
            top = x.max(-1, keepdims=True)
            w = np.exp(x - top)
            total = w.sum(-1, keepdims=True)
            r.out[t] = np.einsum("hk,khe->he", w / total, vv)
            r.mag[t] = np.einsum("hk,khe->he", w / total, np.abs(vv))
            r.flat[t] = np.abs(vv).sum(0) / total
            r.lse[t] = (top + np.log(total))[:, 0]
            r.dot[t] = abs(scale) * np.einsum("he,khe->hk", np.abs(q[t]), np.abs(kk)).max(-1)
            r.reach[t] = abs(scale) * np.abs(q[t]).max(-1) * np.abs(kk).sum(-1).max(0)
    return r


def bounds(r: Result, dtype, kv_dtype):
    """How far out and lse may be from the 64-bit result.

    A score is a sum of 192 exact products in fp32: off by at most d = 192 * 2^-23 * sum |q k| *
    scale (each addition at most one fp32 step, as a matrix unit that truncates adds), and with
    fp8 keys and bf16 queries by 2^-39 of the largest |q| per element more.  A weight
    exp(x - max) is then off by a factor e^(2d) and rounded to half a step of bf16 (bf16 keys
    and values) or of fp16 (others), or there by 2^-34 of the largest weight.  The sums over
    `longest` rows add longest * 2^-23 relative to the sum of magnitudes; the sum of the weights
    is off by the same factors without the rounding.  Exponentials and the final scaling are fp32
    operations with errors of a few 2^-22.  The result is rounded once: half a step of its
    format, or half of fp16's smallest, 2^-25.  lse is off by d, the relative error of the sum,
    and fp32 roundings of itself."""
    d = 192 * 2.0 ** -23 * r.dot
    if kv_dtype in FP8:
        d = d + 2.0 ** -39 * r.reach
    half16 = dtype is torch.bfloat16 and kv_dtype is torch.bfloat16
    weight = HALF[torch.bfloat16] if half16 else HALF[torch.float16]
    rel = (weight + 4 * d + 2 * r.longest * 2.0 ** -23 + 2.0 ** -18)[..., None]
    err = rel * r.mag + (0.0 if half16 else 2.0 ** -34 * r.flat)
    o = err + HALF[dtype] * (np.abs(r.out) + err) + (2.0 ** -25 if dtype is torch.float16 else 1e-30)
    le = d + r.longest * 2.0 ** -23 + 2.0 ** -18 + \
        2.0 ** -22 * np.abs(np.where(np.isfinite(r.lse), r.lse, 0))
    return o, le


# ------------------------------------------------------------------------ trees
def tree_masks(sizes, seed, words=None):
    """Random ancestor masks (own bit included): bool [T, largest size]."""
    rng = np.random.default_rng(seed)
    width = 32 * words if words else max(sizes)
    rows = []
    for n in sizes:
        m = np.zeros((n, width), bool)
        for i in range(n):
            up = int(rng.integers(-1, i)) if rng.random() < 0.6 else i - 1
            if up >= 0:
                m[i] = m[up]
            if i < width:
                m[i, i] = True
        rows.append(m)
    return np.concatenate(rows) if rows else np.zeros((0, width), bool)


def words_of(masks):
    """The bit words of bool masks: int32 [T, W]."""
    T, n = masks.shape
    pad = np.zeros((T, (n + 31) // 32 * 32), bool)
    pad[:, :n] = masks
    return np.packbits(pad.reshape(T, -1, 32), axis=-1, bitorder="little").view("<u4")[..., 0] \
        .astype(np.uint32).view(np.int32)
