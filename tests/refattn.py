"""Inputs and 64-bit references for the serving operators' tests: the latent
attention, the merge of attention states and the block copies.

``attention`` is the definition in numpy float64 (pinned against the C oracle's
loops by test_oracle_serving.py); ``attention_bounds`` derives how far a result
may be from it.
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


@dataclass
class Result:
    """The definition's result in float64 and what its error bounds need; tokens of no
    sequence are NaN in all."""
    out: np.ndarray    # [T, H, 512]
    lse: np.ndarray    # [T, H]
    mag: np.ndarray    # [T, H, 512]: sum of weight * |row| / sum of weights
    flat: np.ndarray   # [T, H, 512]: sum of |row| / sum of weights (the largest weight is 1)
    dot: np.ndarray    # [T, H]: largest |scale| * sum |q row|
    reach: np.ndarray  # [T, H]: largest |scale| * max |q| * sum |row|
    longest: int
    fp8: bool


def attention(pg: Paged, q, cu, kv_lens, scale=SCALE, causal=True) -> Result:
    T, H, _ = q.shape
    qv = orc.bf16_bits_to_f64(q).reshape(q.shape)
    wide, flat2 = (T, H, RANK), (T, H)
    r = Result(*(np.full(sh, np.nan) for sh in (wide, flat2, wide, wide, flat2, flat2)),
               max(1, max(int(k) for k in kv_lens)), pg.fmt != 0)
    for s, kv in enumerate(kv_lens):
        a, b = int(cu[s]), min(int(cu[s + 1]), T)
        n = int(cu[s + 1]) - a
        if b <= a:
            continue
        rows, found = rows_of(pg, s, max(0, int(kv)))
        for t in range(a, b):
            seen = max(0, int(kv) - n + 1 + t - a if causal else int(kv))
            k = rows[:seen][found[:seen]]
            for x in (r.out, r.mag, r.flat, r.dot, r.reach):
                x[t] = 0.0
            r.lse[t] = -np.inf
            if len(k) == 0:
                continue
            x = scale * (qv[t] @ k.T)
            top = x.max(-1, keepdims=True)
            w = np.exp(x - top)
            total = w.sum(-1, keepdims=True)
            v = np.abs(k[:, :RANK])
            with np.errstate(invalid="ignore"):
                r.out[t], r.mag[t] = (w / total) @ k[:, :RANK], (w / total) @ v
            r.flat[t] = v.sum(0) / total
            r.lse[t] = (top + np.log(total))[:, 0]
            r.dot[t] = abs(scale) * (np.abs(qv[t]) @ np.abs(k).T).max(-1)
            r.reach[t] = abs(scale) * np.abs(qv[t]).max(-1) * np.abs(k).sum(-1).max()
    return r


def attention_bounds(r: Result):
    """How far out and lse may be from the float64 result.

    A score is a sum of 576 exact products in fp32: off by at most d = 576 * 2^-23
    * sum |q row| * scale (each addition at most one fp32 step, as a matrix unit
    that truncates adds).  With an fp8 cache the query is two e4m3 parts of itself
    times a power of two that puts its largest value into [2^7, 2^8): exact, or off
    by half the second part's smallest step, 2^-10 / 16 = 2^-14, that is by 2^-21 of
    the largest value at most, so d grows by 2^-21 * scale * max |q| * sum |row|.
    A weight exp(x - max) is then off by a factor e^(2d) (its score and the
    maximum) and rounded to 8 bits: by 2^-8 of itself; as two e4m3 parts with an fp8
    cache by 2^-8 (2^-4 each) or, below the second part's smallest step / 512, by
    2^-19 of the unit that weights are relative to, which is at most the largest
    weight (the reference maximum is never above the true one).  The sums over
    `longest` rows add longest * 2^-23 relative to the sum of magnitudes; the sum of
    the weights is off by the same factors without the rounding to 8 bits.  The
    result is rounded once to bf16 (2^-8 of its value).  Exponentials and the final
    scaling are fp32 operations with errors of a few 2^-22.
    lse is off by d, the relative error of the sum, and fp32 roundings of itself."""
    d = 576 * 2.0 ** -23 * r.dot
    part = 0.0
    if r.fp8:
        d = d + 2.0 ** -21 * r.reach
        part = 2.0 ** -19 * r.flat
    rel = (BF16_HALF + 4 * d + 2 * r.longest * 2.0 ** -23 + 2.0 ** -18)[..., None]
    err = rel * r.mag + part
    o = err + BF16_HALF * (np.abs(r.out) + err) + 1e-30
    le = d + r.longest * 2.0 ** -23 + 2.0 ** -18 + \
        4 * FP32_HALF * np.abs(np.where(np.isfinite(r.lse), r.lse, 0))
    return o, le
