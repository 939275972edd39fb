"""GPU parity of mla_latent_tree_attention with its definition in 64 bits, within
refattn.attention_bounds: trees of different sizes, masks that name nothing, rows that no mask
names, masks shorter and longer than the trees, and what surrounds the data."""
import numpy as np
import pytest
import torch

import devutil as D
import refattn as R
import refprefill as P
from pack_mla_cache_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pack_mla_cache_gb300 import build
    build.build()
    ops.lib()


def expected(pg, q, cu, kv_lens, masks, scale=R.SCALE):
    """refattn.attention with a token's rows chosen by its mask."""
    T, H, _ = q.shape
    qv = R.orc.bf16_bits_to_f64(q).reshape(q.shape)
    wide, flat2 = (T, H, R.RANK), (T, H)
    r = R.Result(*(np.full(s, np.nan) for s in (wide, flat2, wide, wide, flat2, flat2)),
                 max(1, max(int(k) for k in kv_lens)), pg.fmt != 0)
    for s, kv in enumerate(kv_lens):
        n = cu[s + 1] - cu[s]
        if n <= 0:
            continue
        rows, found = R.rows_of(pg, s, max(0, int(kv)))
        for t in range(cu[s], min(cu[s + 1], T)):
            see = found.copy()
            for p in range(max(0, kv - n), kv):
                i = p - (kv - n)
                see[p] &= bool(i < masks.shape[1] and masks[t, i])
            k = rows[see]
            for x in (r.out, r.mag, r.flat, r.dot, r.reach):
                x[t] = 0.0
            r.lse[t] = -np.inf
            if len(k) == 0:
                continue
            x = scale * (qv[t] @ k.T)
            top = x.max(-1, keepdims=True)
            w = np.exp(x - top)
            total = w.sum(-1, keepdims=True)
            v = np.abs(k[:, :R.RANK])
            r.out[t], r.mag[t] = (w / total) @ k[:, :R.RANK], (w / total) @ v
            r.flat[t] = v.sum(0) / total
            r.lse[t] = (top + np.log(total))[:, 0]
            r.dot[t] = abs(scale) * (np.abs(qv[t]) @ np.abs(k).T).max(-1)
            r.reach[t] = abs(scale) * np.abs(qv[t]).max(-1) * np.abs(k).sum(-1).max()
    return r


class Call:
    def __init__(self, pg, q, cu, kv, masks, *, mask_pad=0, cache=None):
        T, H, _ = q.shape
        self.pg, self.cu, self.kv, self.masks, self.qh = pg, cu, kv, masks, q
        self.q = D.dev_bf16(q)
        self.cache = cache if cache is not None else D.dev_bf16(pg.cache) if pg.fmt == 0 else D.dev(pg.cache)
        self.k_scale = None if pg.k_scale is None else torch.tensor([pg.k_scale], device="cuda")
        self.table = D.dev(pg.table)
        w = P.words_of(masks)
        wide = np.full((T, w.shape[1] + mask_pad), -1, np.int32)
        wide[:, :w.shape[1]] = w
        self.mask = D.dev(wide)[:, :w.shape[1]]
        self.cu_t, self.kv_t = D.dev(np.asarray(cu, np.int32)), D.dev(np.asarray(kv, np.int32))
        self.out = torch.full((T, H, R.RANK), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((T, H), 7.0, device="cuda")
        n = ops.mla_latent_attention_workspace(T, H, len(kv))
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, **kw):
        pg = self.pg
        ops.mla_latent_tree_attention(self.q[:, :, :512], self.q[:, :, 512:], self.cache, pg.fmt,
                                      pg.num_blocks, pg.block, pg.block_stride, pg.entry_stride,
                                      self.table, self.cu_t, self.kv_t, self.mask, self.out, self.ws,
                                      softmax_scale=R.SCALE, k_scale=self.k_scale, lse=self.lse,
                                      err_word=self.err, **kw)
        return self

    def got(self):
        torch.cuda.synchronize()
        return P.f64(self.out.cpu()), P.f64(self.lse.cpu()), int(self.err.item())

    def check(self, err=0):
        out, lse, e = self.got()
        r = expected(self.pg, self.qh, self.cu, self.kv, self.masks)
        own = ~np.isnan(r.lse)
        assert (out[~own] == 7).all() and (lse[~own] == 7).all()
        none = np.isneginf(r.lse)
        assert (out[none] == 0).all() and np.isneginf(lse[none]).all()
        bo, bl = R.attention_bounds(r)
        live = own & ~none
        assert np.isfinite(out[live]).all() and np.isfinite(lse[live]).all()
        if live.any():
            worst = (np.abs(out[live] - r.out[live]) / bo[live]).max()
            worst_l = (np.abs(lse[live] - r.lse[live]) / bl[live]).max()
            assert worst <= 1 and worst_l <= 1, (worst, worst_l)
        assert e == err
        return self


def cu_of(n):
    return [0] + [int(x) for x in np.cumsum(n)]


CASES = [
    # tree sizes, cache rows (new ones included), heads, cache, block
    ([1], [1], 1, 0, 64), ([8], [8], 16, 0, 64), ([8], [300], 16, 1, 16), ([7, 1, 16], [64, 130, 500], 16, 2, 16),
    ([31, 33, 64], [95, 700, 64], 8, 0, 64), ([5, 0, 9], [60, 40, 9], 40, 1, 1), ([61, 61], [1000, 63], 16, 0, 48),
    ([100], [2100], 3, 1, 100), ([130, 4], [131, 5000], 5, 0, 64), ([12], [9000], 128, 1, 128),
    ([16] * 5, [90, 700, 16, 17, 3000], 16, 1, 64), ([4, 4], [4, 66], 128, 0, 7),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_parity(case):
    n, kv, heads, fmt, block = case
    pg = R.paged(kv, fmt, block, seed=5)
    q = R.queries(sum(n), heads)
    Call(pg, q, cu_of(n), kv, P.tree_masks(n, 3), mask_pad=3).run().check()


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_any_masks(fmt):
    """Masks that name nothing, later rows, everything; with and without context; more tokens than
    rows (the first tokens' rows do not exist)."""
    n, kv = [20, 40, 33, 9], [20, 140, 12, 0]
    pg = R.paged(kv, fmt, 16, seed=8)
    masks = np.random.default_rng(2).random((sum(n), 40)) < 0.2
    masks[0] = masks[25] = masks[70] = False
    masks[3] = masks[30] = masks[62] = True
    Call(pg, R.queries(sum(n), 16), cu_of(n), kv, masks).run().check()


@pytest.mark.parametrize("words", [1, 2, 5])
def test_mask_widths(words):
    """Rows whose words lie behind the mask are not seen; words behind the tree change nothing."""
    n, kv = [70, 12], [200, 80]
    pg = R.paged(kv, 1, 64, seed=9)
    masks = P.tree_masks(n, 4, words=words)
    masks[:, 90:] = True
    Call(pg, R.queries(82, 16), cu_of(n), kv, masks, mask_pad=1).run().check()


@pytest.mark.parametrize("seed", range(20))
def test_random_batches(seed):
    rng = np.random.default_rng(500 + seed)
    s = int(rng.integers(1, 10))
    heads = int(rng.choice([1, 2, 8, 16, 16, 33, 64, 128]))
    n = [int(rng.choice([0, 1, 2, 8, int(rng.integers(1, max(2, min(80, 1200 // heads // s)) + 1))])) for _ in range(s)]
    n[0] = max(n[0], 1)
    kv = [x + int(rng.choice([0, 1, 63, 64, 65, int(rng.integers(0, 2000 // s))])) for x in n]
    pg = R.paged(kv, int(rng.integers(0, 3)), int(rng.choice([1, 8, 16, 24, 64, 128])), seed=seed)
    Call(pg, R.queries(sum(n), heads, seed=seed), cu_of(n), kv, P.tree_masks(n, seed)).run().check()


@pytest.mark.parametrize("fmt", [0, 1])
def test_a_chain_is_the_causal_attention(fmt):
    """A tree of one branch gives the bits of mla_latent_attention."""
    n, kv, H = [5, 9, 1], [300, 9, 700], 16
    pg = R.paged(kv, fmt, 64)
    q = R.queries(sum(n), H)
    masks = np.concatenate([np.tril(np.ones((x, 9), bool)) for x in n])
    c = Call(pg, q, cu_of(n), kv, masks).run()
    out, lse, _ = c.got()
    ops.mla_latent_attention(c.q[:, :, :512], c.q[:, :, 512:], c.cache, pg.fmt, pg.num_blocks, pg.block,
                             pg.block_stride, pg.entry_stride, c.table, c.cu_t, c.kv_t, c.out, c.ws,
                             softmax_scale=R.SCALE, k_scale=c.k_scale, lse=c.lse, causal=True)
    o2, l2, _ = c.got()
    # the cut over the SMs differs (first tokens see fewer rows): fp32 roundings, then one to bf16
    r = expected(pg, q, cu_of(n), kv, masks)
    bo, bl = R.attention_bounds(r)
    assert (np.abs(out - o2) <= 2 * bo).all() and (np.abs(lse - l2) <= 2 * bl).all()


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_bad_rows_stay_unseen(fmt):
    """A new row with a NaN is felt by the tokens whose masks name it, and by no other."""
    n, kv = [10], [100]
    pg = R.paged(kv, fmt, 16, seed=3)
    q, masks = R.queries(10, 16), P.tree_masks(n, 7)
    masks[6, 4] = True
    masks[7:, 4] = False
    clean = Call(pg, q, [0, 10], kv, masks).run().got()
    c = Call(pg, q, [0, 10], kv, masks)
    p = 90 + 4
    blk = int(pg.table[0, p // 16])
    at = blk * pg.block_stride + (p % 16) * pg.entry_stride
    flat = c.cache.view(-1).view(torch.int16 if fmt == 0 else torch.uint8)
    flat[at + 3:at + 9] = 0x7FC0 if fmt == 0 else 0x7F
    out, lse, _ = c.run().got()
    sees = masks[:, 4]
    assert np.isnan(out[sees]).all() and np.array_equal(out[~sees], clean[0][~sees])
    assert np.array_equal(lse[~sees], clean[1][~sees])


def test_missing_block_and_unowned_tokens():
    n, kv = [6, 6], [130, 40]
    pg = R.paged(kv, 0, 16, seed=6)
    pg.table[0, 2] = -7
    q, masks = R.queries(14, 16), P.tree_masks([14], 1)
    Call(pg, q, [1, 7, 13], kv, masks).run().check(err=ops.MLA_ERRBIT_BLOCK_OOB)


def test_streams_and_graphs_repeat_to_the_bit():
    n, kv = [16] * 4, [900, 33, 16, 4000]
    pg = R.paged(kv, 1, 64)
    c = Call(pg, R.queries(64, 16), cu_of(n), kv, P.tree_masks(n, 2)).run()
    first = c.got()
    c.out.fill_(3.0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for _ in range(3):
        g.replay()
    again = c.got()
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])
    c.out.fill_(3.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    s.synchronize()
    assert np.array_equal(first[0], c.got()[0])


def test_masks_past_32_bits():
    """Mask rows 2 GB apart."""
    n, kv = [3], [70]
    pg = R.paged(kv, 0, 16)
    c = Call(pg, R.queries(3, 16), cu_of(n), kv, P.tree_masks(n, 4))
    big = torch.empty(2 * (1 << 29) + 8, dtype=torch.int32, device="cuda")
    far = big.as_strided(tuple(c.mask.shape), (1 << 29, 1))
    far.copy_(c.mask)
    c.mask = far
    c.run().check()


def test_device_refusals():
    n, kv = [3], [70]
    c = Call(R.paged(kv, 0, 16), R.queries(3, 16), cu_of(n), kv, P.tree_masks(n, 4))
    ws = c.ws
    c.ws = ws[:-16]
    with pytest.raises(ops.MlaError, match="workspace_bytes must be >="):
        c.run()
    c.ws = ws
    c.mask = c.mask.cpu()
    with pytest.raises(ops.MlaError, match="tree_mask must be device memory"):
        c.run()


@pytest.mark.parametrize("stage", [1, 2])
@pytest.mark.parametrize("fmt,heads", [(0, 16), (1, 16), (0, 128)])
def test_waits_that_run_out_return_and_report(fmt, heads, stage):
    """With a 1 ms limit and a pipeline stage of the first CTA that never fills (a testing hook),
    its waits run out: the call returns and says so, the other CTAs' sequences are as ever, and
    the next call is exact.  No fault is involved: only bounded waits that give up."""
    n = [2] * 200
    kv = [1500] + [64 * (i % 5 + 1) for i in range(199)]
    pg = R.paged(kv, fmt, 64, seed=19)
    c = Call(pg, R.queries(400, heads), cu_of(n), kv, P.tree_masks(n, 4)).run()
    good = c.got()[0]
    c.out.fill_(3.0)
    torch.cuda.synchronize()
    try:
        ops.mla_test_attention_timeout(1_000_000, stage)
        out, _, e = c.run().got()
    finally:
        ops.mla_test_attention_timeout()
    assert e == ops.MLA_ERRBIT_TIMEOUT
    assert np.array_equal(out[80:], good[80:]) and not np.array_equal(out[:2], good[:2])
    c.err.zero_()
    out, _, e = c.run().got()
    assert e == 0 and np.array_equal(out, good)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_bad_queries_that_see_no_row(fmt, bad):
    """A token whose mask names nothing and that has no context has 0 and -infinity, whatever its
    query holds; the others are as ever."""
    n = [12, 30]
    pg = R.paged(n, fmt, 16, seed=8)
    masks = P.tree_masks(n, 2)
    none = np.zeros(42, bool)
    none[[0, 5, 11, 12, 13, 14, 15, 40]] = True
    masks[none] = False
    q = R.queries(42, 16)
    c = Call(pg, q, cu_of(n), n, masks).run().check()
    want = c.got()
    c.q[torch.from_numpy(none).cuda()] = bad
    out, lse, e = c.run().got()
    assert np.array_equal(out, want[0]) and np.array_equal(lse, want[1]) and e == 0


def _times(pg, s, p, mul):
    """Row p of sequence s of a paged cache times a factor, cut to what the format holds."""
    o = int(pg.table[s, p // pg.block]) * pg.block_stride + (p % pg.block) * pg.entry_stride
    row = pg.cache[o:o + R.ENTRY]
    if pg.fmt == 0:
        pg.cache[o:o + R.ENTRY] = R.orc.bf16_from_f32_array((R.orc.bf16_bits_to_f64(row) * mul).astype(np.float32))
    else:
        x = np.clip(R.orc.fp8_decode(row, pg.fmt).astype(np.float32) * np.float32(mul), -440, 440)
        pg.cache[o:o + R.ENTRY] = R.orc.fp8_encode(x, pg.fmt)


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("heads", [1, 4, 16])
def test_a_large_row_moves_no_token_that_does_not_name_it(fmt, heads):
    """The masks of every other token name a drafted row whose scores dwarf the others; the tokens
    between, rows of the same query tile, keep every bit.  The row lies behind tiles of smaller
    ones, so its readers' references have to move; enough sequences (over the same blocks) that most
    are not cut in front of it."""
    S, n, ctx = 300, 8, 200
    masks = P.tree_masks([n] * S, 3)
    masks[:, 4] = np.arange(S * n) % 2 == 1
    got = []
    for mul in (1.0, 20.0):
        pg = R.paged([ctx + n], fmt, 64, seed=4)
        for p in range(192):
            _times(pg, 0, p, 0.5)
        _times(pg, 0, ctx + 4, mul)
        pg.table = np.repeat(pg.table, S, 0)
        c = Call(pg, R.queries(S * n, heads, mul=2.0), cu_of([n] * S), [ctx + n] * S, masks).run()
        got.append(c.got())
        assert got[-1][2] == 0
        if mul > 1:
            c.check()
    sees = masks[:, 4]
    for a, b in zip(got[0][:2], got[1][:2]):
        assert np.array_equal(a[~sees], b[~sees])
    assert not np.array_equal(got[0][1][sees], got[1][1][sees])


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("case", [([5, 9, 1], [300, 9, 700], 16), ([1] * 40, list(range(1, 2400, 60)), 16),
                                  ([64, 3], [1200, 5000], 4)], ids=["short", "single", "long"])
def test_chains_meet_the_definition_both_ways(fmt, case):
    """Trees of one branch by masks and as causal tokens: each within the bound of the one definition."""
    n, kv, H = case
    pg = R.paged(kv, fmt, 64)
    q = R.queries(sum(n), H)
    masks = np.concatenate([np.tril(np.ones((x, max(n)), bool)) for x in n])
    c = Call(pg, q, cu_of(n), kv, masks).run().check()
    c.out.fill_(7.0)
    c.lse.fill_(7.0)
    ops.mla_latent_attention(c.q[:, :, :512], c.q[:, :, 512:], c.cache, pg.fmt, pg.num_blocks, pg.block,
                             pg.block_stride, pg.entry_stride, c.table, c.cu_t, c.kv_t, c.out, c.ws,
                             softmax_scale=R.SCALE, k_scale=c.k_scale, lse=c.lse, causal=True)
    c.check()
