"""GPU parity of mla_latent_attention with the float64 definition, within
bounds derived in refattn.attention_bounds: types, head counts, lengths from no
row to split contexts, page sizes, strides, masks, and what surrounds the data
(NaN rows behind a sequence and in rows a token does not see, unowned tokens,
bad block ids); streams, graphs and repeated calls give the same bits."""
import numpy as np
import pytest
import torch

import devutil as D
import refattn as R
from pack_mla_cache_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pack_mla_cache_gb300 import build
    build.build()
    ops.lib()


def dev_cache(pg):
    return D.dev_bf16(pg.cache) if pg.fmt == 0 else D.dev(pg.cache)


def workspace(T, H, S):
    n = ops.mla_latent_attention_workspace(T, H, S)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN words


class Call:
    """One call's device buffers; out and lse start as canaries."""

    def __init__(self, pg, q, cu, kv, *, causal=True, scale=R.SCALE, cache=None, pad=0):
        T, H, _ = q.shape
        self.pg, self.cu, self.kv, self.causal, self.scale = pg, cu, kv, causal, scale
        qs = np.zeros((T, H + (1 if pad else 0), R.ENTRY + pad), np.uint16)
        qs[:, :H, :R.ENTRY] = q
        self.q = D.dev_bf16(qs)[:, :H]
        self.cache = dev_cache(pg) if cache is None else cache
        self.k_scale = None if pg.k_scale is None else torch.tensor([pg.k_scale], device="cuda")
        self.table = D.dev(pg.table)
        self.cu_t, self.kv_t = D.dev(np.asarray(cu, np.int32)), D.dev(np.asarray(kv, np.int32))
        self.out_full = torch.full((T + 1, H + (1 if pad else 0), R.RANK + pad), 7.0,
                                   dtype=torch.bfloat16, device="cuda")
        self.out = self.out_full[:T, :H, :R.RANK]
        self.lse_full = torch.full((H + 1, T + 1), 7.0, device="cuda") if pad else \
            torch.full((T + 1, H), 7.0, device="cuda")
        self.lse = (self.lse_full.t() if pad else self.lse_full)[:T, :H]
        self.ws = workspace(T, H, len(kv))
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, **kw):
        pg, q = self.pg, self.q
        ops.mla_latent_attention(q[:, :, :512], q[:, :, 512:576], self.cache, pg.fmt,
                                 pg.num_blocks, pg.block, pg.block_stride, pg.entry_stride,
                                 self.table, self.cu_t, self.kv_t, self.out, self.ws,
                                 **{**dict(softmax_scale=self.scale, k_scale=self.k_scale,
                                           causal=self.causal, lse=self.lse, err_word=self.err),
                                    **kw})
        return self

    def got(self):
        torch.cuda.synchronize()
        return (self.out.float().cpu().numpy().astype(np.float64),
                self.lse.cpu().numpy().astype(np.float64), int(self.err.item()))

    def canaries(self):
        T, H = self.out.shape[:2]
        o, le = self.out_full.float().cpu().numpy(), self.lse_full.cpu().numpy()
        assert (o[T:] == 7).all() and (o[:, H:] == 7).all() and (o[:, :, R.RANK:] == 7).all()
        if le.shape[0] == T + 1 and le.shape[1] == H:
            assert (le[T] == 7).all()
        else:
            assert (le[H] == 7).all() and (le[:, T] == 7).all()


def check(call, q, err=0):
    out, lse, e = call.got()
    r = R.attention(call.pg, q, call.cu, call.kv, call.scale, call.causal)
    ro, rl = r.out, r.lse
    own = ~np.isnan(rl)
    assert (out[~own] == 7).all() and (lse[~own] == 7).all()  # unowned tokens are untouched
    none = np.isneginf(rl)
    assert (out[none] == 0).all() and np.isneginf(lse[none]).all()
    bo, bl = R.attention_bounds(r)
    live = own & ~none
    assert np.isfinite(out[live]).all() and np.isfinite(lse[live]).all()
    worst = (np.abs(out[live] - ro[live]) / bo[live]).max() if live.any() else 0
    worst_l = (np.abs(lse[live] - rl[live]) / bl[live]).max() if live.any() else 0
    assert worst <= 1 and worst_l <= 1, (worst, worst_l)
    call.canaries()
    assert e == err


def cu_of(q_lens):
    return [0] + list(np.cumsum(q_lens))


CASES = [
    # kv_lens, q_lens, heads, cache, block, causal
    ([1], [1], 1, 0, 64, True),
    ([64], [1], 16, 0, 64, True),
    ([63, 65, 128, 1], [1, 1, 1, 1], 16, 0, 64, True),
    ([500], [1], 16, 1, 16, True),
    ([129, 0, 700], [1, 1, 1], 3, 2, 48, True),
    ([333, 17], [1, 1], 40, 1, 1, True),
    ([257], [1], 128, 0, 64, True),
    ([1000, 90], [1, 1], 128, 1, 128, True),
    ([70, 300, 4], [4, 4, 4], 16, 2, 16, True),
    ([70, 300, 4], [4, 2, 4], 8, 0, 32, True),
    ([300, 200], [100, 37], 16, 0, 64, True),
    ([300, 200], [100, 37], 16, 1, 100, True),
    ([130, 3], [130, 5], 5, 2, 64, True),          # prefill without context; more tokens than rows
    ([260, 50, 20], [70, 1, 20], 24, 0, 64, False),
    ([33, 2000, 1, 0, 512], [3, 1, 1, 0, 2], 17, 1, 64, True),   # a sequence without tokens
    ([5000], [1], 16, 0, 64, True),                # split over many CTAs
    ([4097, 100, 3001], [2, 1, 1], 16, 1, 64, True),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_parity(case):
    kv, ql, heads, fmt, block, causal = case
    pg = R.paged(kv, fmt, block, seed=11)
    q = R.queries(sum(ql), heads)
    check(Call(pg, q, cu_of(ql), kv, causal=causal).run(), q)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("block", [1, 7, 8, 16, 24, 40, 64, 96, 128, 256])
def test_page_sizes(fmt, block):
    """Pages that are parts of a tile, tiles, several tiles, and neither; one page missing."""
    kv, ql = [391, 64, 200], [1, 2, 1]
    pg = R.paged(kv, fmt, block, seed=block)
    if pg.table.shape[1] > 2:
        pg.table[2, 1] = -5
    q = R.queries(4, 16)
    missing = kv[2] > block
    check(Call(pg, q, cu_of(ql), kv).run(), q, err=ops.MLA_ERRBIT_BLOCK_OOB if missing else 0)


@pytest.mark.parametrize("block", [7, 8, 16, 24, 32, 64])
def test_page_sizes_at_64_query_rows(block):
    """The widest query tiles take a stage in halves: pages of every size, a page missing, mixed
    tiles of a few new tokens, two query tiles per sequence."""
    kv, ql = [391, 64, 1000, 130], [1, 2, 3, 1]
    pg = R.paged(kv, 0, block, seed=block)
    pg.table[2, 3] = pg.num_blocks
    q = R.queries(7, 96)
    check(Call(pg, q, cu_of(ql), kv).run(), q, err=ops.MLA_ERRBIT_BLOCK_OOB)


@pytest.mark.parametrize("seed", range(30))
def test_random_batches(seed):
    """Batches of every mixture: head counts, new tokens, lengths around the tile and
    split borders, pages, types, both masks."""
    rng = np.random.default_rng(1000 + seed)
    n = int(rng.integers(1, 12))
    heads = int(rng.choice([1, 2, 5, 8, 16, 16, 31, 33, 64, 100, 128]))
    most = max(1, 1500 // heads // n)
    ql = [int(rng.choice([0, 1, 1, 1, 2, int(rng.integers(1, most + 1))])) for _ in range(n)]
    ql[0] = max(ql[0], 1)
    kv = [int(rng.choice([0, 1, 63, 64, 65, 128, int(rng.integers(1, 300)),
                          int(rng.integers(1, 4000 // n + 2))])) for _ in range(n)]
    fmt, block = int(rng.integers(0, 3)), int(rng.choice([8, 16, 32, 48, 64, 128]))
    pg = R.paged(kv, fmt, block, seed=seed, pad_entry=int(rng.choice([0, 16])))
    q = R.queries(sum(ql), heads, seed=seed, mul=float(rng.choice([0.3, 1.0, 4.0])))
    check(Call(pg, q, cu_of(ql), kv, causal=bool(rng.integers(0, 2))).run(), q)


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_query_magnitudes(fmt):
    """Rows of very different sizes, and rows whose elements are (an fp8 cache takes
    the query in two 4-bit parts relative to the row's largest)."""
    pg = R.paged([300], fmt, 64)
    q = R.orc.bf16_bits_to_f64(R.queries(1, 16))
    q[0, 0] *= 1e-30
    q[0, 1] *= 2.0 ** -100
    q[0, 2] *= 30
    q[0, 3, ::7] *= 100
    q[0, 4] *= np.exp(np.linspace(-12, 1, R.ENTRY))
    q[0, 5] = 0
    q[0, 6] = 0
    q[0, 6, 575] = 8
    q = R.orc.bf16_from_f32_array(q.astype(np.float32))
    check(Call(pg, q, [0, 1], [300]).run(), q)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("bad", [0x7FC0, 0x7F80, 0xFF80])
def test_a_bad_query_row_stays_alone(fmt, bad):
    pg = R.paged([300], fmt, 64)
    q = R.queries(2, 16)
    good = Call(pg, q, [0, 2], [300]).run().got()
    q[1, 5, 100] = bad
    out, lse, _ = Call(pg, q, [0, 2], [300]).run().got()
    assert np.isnan(out[1, 5]).all() and np.isnan(lse[1, 5])
    keep = np.ones((2, 16), bool)
    keep[1, 5] = False
    assert (out[keep] == good[0][keep]).all() and (lse[keep] == good[1][keep]).all()


def test_negative_lengths_are_empty():
    pg = R.paged([100, 50], 0, 64)
    q = R.queries(2, 16)
    call = Call(pg, q, [0, 1, 2], [0, 50])
    call.kv_t[0] = -3
    check(call.run(), q)


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_strides_and_padding(fmt):
    kv, ql = [150, 77], [9, 1]
    pg = R.paged(kv, fmt, 32, pad_entry=16, pad_block=64)
    q = R.queries(sum(ql) + 2, 6)  # two tokens behind the last sequence
    check(Call(pg, q, cu_of(ql), kv, pad=8).run(), q)


def test_tokens_before_the_first_sequence_are_untouched():
    pg = R.paged([50], 0, 64)
    q = R.queries(5, 4)
    check(Call(pg, q, [2, 3], [50]).run(), q)


def test_tokens_past_num_tokens_are_not_computed():
    pg = R.paged([50, 20], 0, 64)
    q = R.queries(4, 4)
    check(Call(pg, q, [0, 2, 9], [50, 20]).run(), q)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("mul,scale", [(16.0, R.SCALE), (1.0, -R.SCALE), (1.0, 0.0)])
def test_score_ranges(fmt, mul, scale):
    """Large scores (the maximum moves far while the rows pass), negative and zero scales."""
    kv, ql = [700, 321], [1, 20]
    pg = R.paged(kv, fmt, 64)
    q = R.queries(sum(ql), 16, mul=mul)
    check(Call(pg, q, cu_of(ql), kv, scale=float(np.float32(scale))).run(), q)


@pytest.mark.parametrize("fmt", [0, 1])
def test_growing_scores(fmt):
    """Every row scores higher than the one before, so the maximum grows throughout."""
    n = 640
    pg = R.paged([n], fmt, 64)
    rng = np.random.default_rng(3)
    base = rng.standard_normal(R.ENTRY)
    x = (base[None] * np.linspace(-1, 1, n)[:, None] * 2).astype(np.float32)
    codes = R.orc.bf16_from_f32_array(x) if fmt == 0 else \
        R.orc.fp8_encode(x / np.float32(pg.k_scale), fmt)
    for p in range(n):
        o = int(pg.table[0, p // 64]) * pg.block_stride + (p % 64) * pg.entry_stride
        pg.cache[o:o + R.ENTRY] = codes[p]
    q = np.repeat(R.orc.bf16_from_f32_array(base.astype(np.float32))[None, None], 16, 1)
    check(Call(pg, np.ascontiguousarray(q), [0, 1], [n]).run(), q)


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_rows_a_token_does_not_see_have_no_influence(fmt):
    """New tokens whose rows hold NaN or infinities: the tokens before them keep
    the result of finite rows."""
    n, ctx, heads = 40, 100, 16
    pg = R.paged([ctx + n], fmt, 64)
    q = R.queries(n, heads)
    call = Call(pg, q, [0, n], [ctx + n]).run()
    good = call.got()
    bad = [0x7FC0, 0x7F80, 0xFF80] if fmt == 0 else [0x7F, 0xFF] if fmt == 1 else [0x7C, 0xFC, 0x7F]
    for j, col in ((17, 5), (25, 570), (33, 100)):
        p = ctx + j
        o = int(pg.table[0, p // 64]) * pg.block_stride + (p % 64) * pg.entry_stride
        pg.cache[o + col] = bad[j % len(bad)]
    out, lse, _ = Call(pg, q, [0, n], [ctx + n]).run().got()
    assert (out[:17] == good[0][:17]).all() and (lse[:17] == good[1][:17]).all()
    assert np.isfinite(out[:17]).all()


def test_bad_block_ids_are_left_out():
    kv, ql = [200, 100], [1, 8]
    pg = R.paged(kv, 1, 16)
    pg.table[0, 3], pg.table[0, 7], pg.table[1, 2] = pg.num_blocks, -1, 1 << 30
    q = R.queries(9, 16)
    check(Call(pg, q, cu_of(ql), kv).run(), q, err=ops.MLA_ERRBIT_BLOCK_OOB)


def test_a_length_beyond_the_table_is_cut():
    pg = R.paged([64], 0, 16, extra_width=0)
    q = R.queries(1, 16)
    call = Call(pg, q, [0, 1], [64], causal=False)
    call.kv_t.fill_(1 << 30)
    call.run()
    check(call, q, err=ops.MLA_ERRBIT_BLOCK_OOB)


def test_every_row_of_a_sequence_invalid():
    pg = R.paged([200], 0, 64)
    pg.table[:] = -1
    q = R.queries(1, 16)
    check(Call(pg, q, [0, 1], [200]).run(), q, err=ops.MLA_ERRBIT_BLOCK_OOB)


def test_no_lse_and_no_error_word():
    pg = R.paged([200], 0, 64)
    q = R.queries(2, 16)
    a, b = Call(pg, q, [0, 2], [200]).run(), Call(pg, q, [0, 2], [200]).run(lse=None, err_word=None)
    assert (a.got()[0] == b.got()[0]).all()
    assert (b.got()[1] == 7).all()


def test_broadcast_query():
    """A query with stride 0 over the heads."""
    pg = R.paged([90], 0, 64)
    q1 = R.queries(1, 1)
    call = Call(pg, np.ascontiguousarray(np.repeat(q1, 8, 1)), [0, 1], [90])
    call.q = D.dev_bf16(q1).expand(1, 8, R.ENTRY)
    check(call.run(), np.repeat(q1, 8, 1))


def test_many_sequences():
    rng = np.random.default_rng(2)
    kv = list(rng.integers(0, 90, 700))
    pg = R.paged(kv, 1, 32)
    q = R.queries(700, 4)
    check(Call(pg, q, cu_of([1] * 700), kv).run(), q)


@pytest.mark.parametrize("n", [31, 32, 33, 63, 96, 97, 128, 129])
def test_batch_sizes_with_empty_sequences(n):
    """Batches of every shape that the CTAs cut their runs from: some sequences have no tokens,
    some no rows, one has several query tiles."""
    rng = np.random.default_rng(n)
    kv = rng.integers(0, 200, n)
    ql = rng.integers(0, 3, n)
    ql[n // 2] = 9
    ql[0], kv[0] = 0, 50
    kv[n - 1] = 700
    pg = R.paged(list(kv), n % 3, 16, seed=n)
    q = R.queries(int(ql.sum()), 8)
    check(Call(pg, q, cu_of([int(x) for x in ql]), [int(x) for x in kv]).run(), q)


def test_most_sequences():
    kv = [1 + (i % 7) for i in range(4096)]
    pg = R.paged(kv, 0, 16)
    q = R.queries(4096, 1)
    check(Call(pg, q, cu_of([1] * 4096), kv).run(), q)


def test_long_context_many_splits():
    n = 33000
    pg = R.paged([n], 1, 64)
    q = R.queries(1, 16)
    check(Call(pg, q, [0, 1], [n]).run(), q)


def test_offsets_past_32_bits():
    """The sequence's blocks lie behind the first 4 GiB (and 2^32 elements) of the cache."""
    pg = R.paged([200], 1, 64)
    far = (1 << 32) // (64 * R.ENTRY) + 5
    big = torch.zeros((far + pg.num_blocks) * 64 * R.ENTRY, dtype=torch.uint8, device="cuda")
    big[far * 64 * R.ENTRY:] = D.dev(pg.cache)
    q = R.queries(3, 16)
    call = Call(pg, q, [0, 3], [200], cache=big)
    call.table = torch.where(call.table >= 0, call.table + far, call.table)
    nb, pg.num_blocks = pg.num_blocks, far + pg.num_blocks
    call.run()
    pg.num_blocks = nb
    check(call, q)


def test_repeated_calls_give_the_same_bits():
    kv, ql = [3000, 517, 64], [1, 30, 5]
    pg = R.paged(kv, 1, 64)
    q = R.queries(sum(ql), 16)
    call = Call(pg, q, cu_of(ql), kv).run()
    a = call.got()
    for _ in range(3):
        b = call.run().got()
        assert (a[0] == b[0]).all() and (a[1] == b[1]).all()


def test_back_to_back_calls_share_a_workspace():
    """Queued without a wait between them, on one workspace, with programmatic
    dependent launch on and off."""
    sets = []
    for seed, (kv, ql) in enumerate([([2500], [1]), ([300, 400], [20, 1]), ([1, 64], [1, 1])]):
        pg = R.paged(kv, seed % 3, 64, seed=seed)
        q = R.queries(sum(ql), 16, seed=seed)
        sets.append((Call(pg, q, cu_of(ql), kv), q))
    ws = max((c.ws for c, _ in sets), key=lambda t: t.numel())
    for c, _ in sets:
        c.ws = ws
    for pdl in (True, False):
        prev = ops.mla_set_pdl(pdl)
        try:
            for c, _ in sets * 4:
                c.run()
        finally:
            ops.mla_set_pdl(prev)
        for c, q in sets:
            check(c, q)


def test_two_streams_with_their_own_workspaces():
    pg = R.paged([2000, 900], 0, 64)
    q = R.queries(2, 16)
    calls = [Call(pg, q, [0, 1, 2], [2000, 900]) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(calls, streams):
            c.run(stream=s)
    for c in calls:
        check(c, q)


def test_captured_and_replayed_with_other_lengths():
    """The lengths are read on the device: a replayed graph follows new ones."""
    pg = R.paged([2000, 900], 1, 64)
    q = R.queries(2, 16)
    call = Call(pg, q, [0, 1, 2], [2000, 900])
    call.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call.run()
    g.replay()
    check(call, q)
    call.kv = [70, 899]
    call.kv_t.copy_(D.dev(np.asarray(call.kv, np.int32)))
    g.replay()
    check(call, q)


def test_refusals_on_the_device():
    pg = R.paged([100], 0, 64)
    q = R.queries(1, 16)
    call = Call(pg, q, [0, 1], [100])
    with pytest.raises(ops.MlaError, match="workspace_bytes"):
        call.ws = call.ws[:-1]
        call.run()
    call = Call(pg, q, [0, 1], [100])
    call.kv_t = call.kv_t.cpu()
    with pytest.raises(ops.MlaError, match="kv_lens must be device memory"):
        call.run()


@pytest.mark.parametrize("stage", [1, 2])
@pytest.mark.parametrize("fmt,heads", [(0, 16), (0, 128), (1, 16), (2, 40)])
def test_waits_that_run_out_return_and_report(fmt, heads, stage):
    """With a 1 ms limit and a pipeline stage of the first CTA that never fills (a testing hook),
    its waits run out: the call returns and says so, the other CTAs' sequences are as ever, and
    the next call is exact.  No fault is involved: only bounded waits that give up."""
    kv = [1500] + [64 * (i % 5 + 1) for i in range(320)]
    pg = R.paged(kv, fmt, 64, seed=19)
    q = R.queries(len(kv), heads)
    cu = list(range(len(kv) + 1))
    good, _, e = Call(pg, q, cu, kv).run().got()
    assert e == 0
    c = Call(pg, q, cu, kv)
    try:
        ops.mla_test_attention_timeout(1_000_000, stage)
        out, _, e = c.run().got()
    finally:
        ops.mla_test_attention_timeout()
    assert e == ops.MLA_ERRBIT_TIMEOUT
    c.canaries()
    np.testing.assert_array_equal(out[40:], good[40:])  # (the first CTA has a few sequences)
    assert not np.array_equal(out[:2], good[:2])
    c.err.zero_()
    out, _, e = c.run().got()
    assert e == 0
    np.testing.assert_array_equal(out, good)


def test_two_graphs_share_a_workspace():
    """Replayed in turn on one stream; each gives its own result every time."""
    calls, want = [], []
    for seed, kv in ((3, [900, 40, 2000]), (4, [70, 1500, 333])):
        pg = R.paged(kv, 1, 64, seed=seed)
        q = R.queries(3, 16, seed=seed)
        calls.append(Call(pg, q, [0, 1, 2, 3], kv))
    calls[1].ws = calls[0].ws
    for c in calls:
        want.append(c.run().got()[:2])
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0, 0):
        calls[i].out.fill_(7.0)
        graphs[i].replay()
        out, lse, e = calls[i].got()
        np.testing.assert_array_equal(out, want[i][0])
        np.testing.assert_array_equal(lse, want[i][1])
        assert e == 0


def test_runs_that_start_and_end_between_query_tiles():
    """Equal short sequences, so that many CTAs' runs begin or end where a query tile does."""
    for n, rows in ((152, 64), (304, 64), (76, 640), (151, 65), (500, 64 * 3)):
        kv = [rows] * n
        pg = R.paged(kv, 1, 64, seed=n)
        q = R.queries(n, 16, seed=n)
        check(Call(pg, q, cu_of([1] * n), kv).run(), q)
