"""Inputs and 64-bit references for the serving operators' tests: the latent
attention, the merge of attention states and the block copies.

``attention`` is the definition in numpy float64 (pinned against the C oracle's
loops by test_oracle_serving.py).  Beside the result it gives what the error
bounds need: per output element the weighted mean of |row|, and per (token,
head) the largest sum of |q * row| * |scale|.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

import oracle as orc

ENTRY, RANK = 576, 512
BF16_HALF, FP16_HALF, FP32_HALF = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24  # eps / 2
SCALE = float(np.float32(192 ** -0.5))  # as the fp32 argument holds it


@dataclass
class Paged:
    """A paged cache of random latent rows and the sequences that own its blocks."""
    cache: np.ndarray        # flat: uint16 (bf16 bits) or uint8 (fp8 codes)
    fmt: int
    num_blocks: int
    block: int
    block_stride: int
    entry_stride: int
    table: np.ndarray        # int32 [S, W]
    k_scale: float | None


def paged(kv_lens, fmt, block, *, seed=0, pad_entry=0, pad_block=0, extra_width=1, k_scale=0.0137):
    """Random rows ~ N(0, 1) (fp8: divided by k_scale) in blocks shuffled over the
    sequences; the padding between entries and blocks and the rows behind each
    sequence hold NaN codes."""
    rng = np.random.default_rng(seed)
    pages = [max(1, -(-int(n) // block)) for n in kv_lens]
    nb = sum(pages) + 2
    es = ENTRY + pad_entry
    bs = block * es + pad_block
    nan = 0x7FC0 if fmt == 0 else 0x7F
    cache = np.full(nb * bs, nan, np.uint16 if fmt == 0 else np.uint8)
    ids = rng.permutation(nb)
    table = np.full((len(pages), max(pages) + extra_width), -7, np.int32)
    at = 0
    for s, n in enumerate(kv_lens):
        table[s, :pages[s]] = ids[at:at + pages[s]]
        at += pages[s]
        x = rng.standard_normal((int(n), ENTRY)).astype(np.float32)
        codes = orc.bf16_from_f32_array(x) if fmt == 0 else \
            orc.fp8_encode(np.clip(x / np.float32(k_scale), -440, 440), fmt)
        for p in range(int(n)):
            o = int(table[s, p // block]) * bs + (p % block) * es
            cache[o:o + ENTRY] = codes[p]
    return Paged(cache, fmt, nb, block, bs, es, table, None if fmt == 0 else k_scale)


def queries(tokens, heads, seed=1, mul=1.0):
    rng = np.random.default_rng(seed)
    return orc.bf16_from_f32_array((mul * rng.standard_normal((tokens, heads, ENTRY))).astype(np.float32))


def rows_of(pg: Paged, s, n):
    """The values of sequence s's first n rows in float64, and which were found."""
    out, found = np.zeros((n, ENTRY)), np.zeros(n, bool)
    lut = None if pg.fmt == 0 else orc.fp8_decode(np.arange(256, dtype=np.uint8), pg.fmt) * \
        float(np.float32(pg.k_scale))
    for p in range(n):
        k = p // pg.block
        if k >= pg.table.shape[1] or not 0 <= pg.table[s, k] < pg.num_blocks:
            continue
        o = int(pg.table[s, k]) * pg.block_stride + (p % pg.block) * pg.entry_stride
        out[p] = orc.bf16_bits_to_f64(pg.cache[o:o + ENTRY]) if pg.fmt == 0 else lut[pg.cache[o:o + ENTRY]]
        found[p] = True
    return out, found


def attention(pg: Paged, q, cu, kv_lens, scale=SCALE, causal=True):
    """(out, lse, mean |row|, largest |scale| * sum |q row|), float64; tokens of
    no sequence are NaN in all."""
    T, H, _ = q.shape
    qv = orc.bf16_bits_to_f64(q).reshape(q.shape)
    out, mag = np.full((T, H, RANK), np.nan), np.full((T, H, RANK), np.nan)
    lse, dot = np.full((T, H), np.nan), np.full((T, H), np.nan)
    for s, kv in enumerate(kv_lens):
        a, b = int(cu[s]), min(int(cu[s + 1]), T)
        n = int(cu[s + 1]) - a
        if b <= a:
            continue
        rows, found = rows_of(pg, s, max(0, int(kv)))
        for t in range(a, b):
            seen = max(0, int(kv) - n + 1 + t - a if causal else int(kv))
            r = rows[:seen][found[:seen]]
            out[t], mag[t], lse[t], dot[t] = 0.0, 0.0, -np.inf, 0.0
            if len(r) == 0:
                continue
            x = scale * (qv[t] @ r.T)
            top = x.max(-1, keepdims=True)
            w = np.exp(x - top)
            total = w.sum(-1, keepdims=True)
            with np.errstate(invalid="ignore"):
                out[t], mag[t] = (w / total) @ r[:, :RANK], (w / total) @ np.abs(r[:, :RANK])
            lse[t] = (top + np.log(total))[:, 0]
            dot[t] = abs(scale) * (np.abs(qv[t]) @ np.abs(r).T).max(-1)
    return out, lse, mag, dot


def attention_bounds(out, lse, mag, dot, longest):
    """How far out and lse may be from the float64 result.

    A score is a sum of 576 exact products in fp32: off by at most d = 576 * 2^-23
    * sum |q row| * scale (each addition at most one fp32 step, as a matrix unit
    that truncates adds).  A weight exp(x - max) is then off by a factor e^(2d)
    (its score and the maximum), rounded once to bf16 (2^-8), and the sums over
    `longest` rows add longest * 2^-23 relative to the sum of magnitudes; the sum
    of the weights is off by the same factors without the bf16 rounding.  The
    result is rounded once to bf16 (2^-8 of its value).  Exponentials and the
    final scaling are fp32 operations with errors of a few 2^-22.
    lse is off by d, the relative error of the sum, and fp32 roundings of itself."""
    d = 576 * 2.0 ** -23 * dot
    rel = (BF16_HALF + 4 * d + 2 * longest * 2.0 ** -23 + 2.0 ** -18)[..., None]
    o = rel * mag + BF16_HALF * (np.abs(out) + rel * mag) + 1e-30
    le = d + longest * 2.0 ** -23 + 2.0 ** -18 + 4 * FP32_HALF * np.abs(np.where(np.isfinite(lse), lse, 0))
    return o, le
