"""GPU parity of mla_prefill_attention with its definition in 64 bits, within the bounds derived
in refprefill.bounds: types, head layouts, lengths from no row to several tiles and cuts, masks,
strides, and what surrounds the data (NaN rows behind a sequence and in rows that a token does
not see, unowned tokens, rows that do not exist); streams, graphs and repeated calls give the
same bits."""
import numpy as np
import pytest
import torch

import refprefill as R
from pack_mla_cache_gb300 import ops

pytestmark = pytest.mark.gpu
BF, HF, E4, E5 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pack_mla_cache_gb300 import build
    build.build()
    ops.lib()


def cu_of(lens):
    return [0] + [int(x) for x in np.cumsum(lens)]


class Call:
    """One call's inputs (on the CPU, changeable before `put`) and device buffers; out and lse
    start as canaries, the workspace as NaN words."""

    def __init__(self, q_lens, kv_lens, heads=2, kv_heads=None, dtype=BF, kv=None, *, causal=True,
                 scale=R.SCALE, seed=0, q_mul=1.5, spare_q=0, spare_kv=0, layout="packed"):
        kv_heads = kv_heads or heads
        self.dtype, self.kv, self.causal, self.scale, self.layout = dtype, kv or dtype, causal, scale, layout
        self.cu_q, self.cu_kv = cu_of(q_lens), cu_of(kv_lens)
        T, K = self.cu_q[-1] + spare_q, self.cu_kv[-1] + spare_kv
        self.q = R.values((T, heads, 192), dtype, seed, q_mul)
        self.key = R.values((K, kv_heads, 192), self.kv, seed + 1, 1.0 if self.kv not in R.FP8 else 30.0)
        if layout == "shared":
            self.key.view(torch.uint8)[:, :, -64 * self.key.element_size():] = \
                self.key.view(torch.uint8)[:, :1, -64 * self.key.element_size():].clone()
        self.v = R.values((K, kv_heads, 128), self.kv, seed + 2, 1.0 if self.kv not in R.FP8 else 30.0)
        self.kv_scale = 0.03 if self.kv in R.FP8 else None

    def put(self):
        T, H, _ = self.q.shape
        K, G, _ = self.key.shape
        raw = lambda t: t.view(torch.uint8)
        es = self.key.element_size()
        self.dq = self.q.cuda()
        if self.layout == "packed":
            key = self.key.cuda()
            self.dk, self.dp, self.dv = key[:, :, :128], key[:, :, 128:], self.v.cuda()
        else:  # kv_b_proj's output with padding behind a row, rotary rows apart
            both = torch.full((K, G, 272 * es), 0xFF, dtype=torch.uint8)
            both[:, :, :128 * es] = raw(self.key[:, :, :128].contiguous())
            both[:, :, 128 * es:256 * es] = raw(self.v)
            both = both.cuda().view(self.kv)
            self.dk, self.dv = both[:, :, :128], both[:, :, 128:256]
            pe = self.key[:, :, 128:].contiguous()
            self.dp = pe[:, 0].contiguous().cuda() if self.layout == "shared" else pe.cuda()
        self.out_full = torch.full((T + 1, H, 136), 7.0, dtype=self.dtype, device="cuda")
        self.out = self.out_full[:T, :, :128]
        self.lse_full = torch.full((H, T + 1), 7.0, device="cuda")
        self.lse = self.lse_full.t()[:T]
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        self.dcq, self.dck = i32(self.cu_q), i32(self.cu_kv)
        self.ds = None if self.kv_scale is None else torch.tensor([self.kv_scale], device="cuda")
        n = ops.mla_prefill_attention_workspace(max(T, 1), H, G, len(self.cu_q) - 1)
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        return self

    def run(self, **kw):
        a = dict(softmax_scale=self.scale, causal=self.causal, kv_scale=self.ds, lse=self.lse,
                 err_word=self.err)
        ops.mla_prefill_attention(self.dq[:, :, :128], self.dq[:, :, 128:], self.dk, self.dp, self.dv,
                                  self.dcq, self.dck, self.out, self.ws, **{**a, **kw})
        return self

    def got(self):
        torch.cuda.synchronize()
        return R.f64(self.out.cpu()), R.f64(self.lse.cpu()), int(self.err.item())

    def expected(self, limit=None):
        ks = 1.0 if self.kv_scale is None else float(np.float32(self.kv_scale))
        key, v = R.f64(self.key) * ks, R.f64(self.v) * ks
        return R.attend(R.f64(self.q), key, v, self.cu_q, self.cu_kv, self.scale, self.causal, limit)

    def check(self, err=0, limit=None):
        out, lse, e = self.got()
        r = self.expected(limit)
        own = ~np.isnan(r.lse)
        assert (out[~own] == 7).all() and (lse[~own] == 7).all()
        none = np.isneginf(r.lse)
        assert (out[none] == 0).all() and np.isneginf(lse[none]).all()
        live = own & ~none
        assert np.isfinite(out[live]).all() and np.isfinite(lse[live]).all()
        bo, bl = R.bounds(r, self.dtype, self.kv)
        if live.any():
            worst = (np.abs(out - r.out)[live] / bo[live]).max()
            worst_l = (np.abs(lse - r.lse)[live] / bl[live]).max()
            assert worst <= 1 and worst_l <= 1, (worst, worst_l)
        full = R.f64(self.out_full.cpu())
        assert (full[-1] == 7).all() and (full[:, :, 128:] == 7).all()
        assert (R.f64(self.lse_full.cpu())[:, -1] == 7).all()
        assert e == err


KINDS = [(BF, BF), (HF, HF), (BF, E4), (BF, E5), (HF, E4), (HF, E5)]


@pytest.mark.parametrize("kind", KINDS, ids=["bf16", "fp16", "bf16-e4m3", "bf16-e5m2", "fp16-e4m3", "fp16-e5m2"])
@pytest.mark.parametrize("lens", [
    ([1], [1]), ([1], [129]), ([5], [0]), ([0, 3, 0], [4, 3, 0]), ([128], [128]), ([127, 129], [127, 129]),
    ([300], [300]), ([1, 2, 1, 1], [77, 256, 1, 900]), ([40, 257], [168, 700]), ([20, 130], [7, 60]),
], ids=str)
def test_types_and_lengths(kind, lens):
    """Causal, among them more tokens than rows (the first ones see nothing)."""
    Call(*lens, heads=2, dtype=kind[0], kv=kind[1]).put().run().check()


@pytest.mark.parametrize("kind", KINDS, ids=str)
@pytest.mark.parametrize("lens", [([1], [1]), ([70], [0]), ([3, 200], [260, 513]), ([129, 1], [127, 1025])], ids=str)
def test_context_without_mask(kind, lens):
    Call(*lens, heads=2, dtype=kind[0], kv=kind[1], causal=False).put().run().check()


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 1), (6, 2), (8, 8), (16, 2), (5, 1), (40, 1), (130, 1), (200, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_head_layouts(heads, kv_heads, causal):
    Call([33, 1, 60], [33, 200, 170], heads, kv_heads, causal=causal).put().run().check()


@pytest.mark.parametrize("kind", [(BF, BF), (HF, HF), (BF, E4)], ids=str)
@pytest.mark.parametrize("layout", ["packed", "apart", "shared"])
def test_layouts(kind, layout):
    """The pack's key, and the kv_b_proj output with NaN behind its rows and k_pe apart."""
    Call([150, 9], [280, 9], 4, 2, kind[0], kind[1], layout=layout).put().run().check()


@pytest.mark.parametrize("kind", [(BF, BF), (HF, HF), (BF, E5)], ids=str)
def test_many_cuts(kind):
    """One sequence and head cut over many blocks, and a batch of very different lengths."""
    Call([1], [9000], 1, dtype=kind[0], kv=kind[1]).put().run().check()
    Call([130], [4000], 1, dtype=kind[0], kv=kind[1]).put().run().check()
    Call([1, 200, 3, 1, 64], [5000, 300, 3, 1, 1000], 2, dtype=kind[0], kv=kind[1]).put().run().check()


@pytest.mark.parametrize("seed", range(30))
def test_random_batches(seed):
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 9))
    kv_heads = int(rng.choice([1, 1, 2, 3]))
    heads = kv_heads * int(rng.choice([1, 1, 2, 3, 7]))
    most = max(2, 2000 // heads // n)
    ql = [int(rng.choice([0, 1, 1, 2, 63, 64, 65, int(rng.integers(1, most + 1))])) for _ in range(n)]
    ql[0] = max(1, ql[0])
    ctx = [int(rng.choice([0, 1, 63, 64, 127, 128, int(rng.integers(0, 1200))])) for _ in range(n)]
    causal = bool(rng.integers(0, 2))
    kind = KINDS[int(rng.integers(0, len(KINDS)))]
    c = Call(ql, [x + (q if causal else 0) for q, x in zip(ql, ctx)], heads, kv_heads, *kind, causal=causal,
             seed=seed, q_mul=float(rng.choice([0.3, 1.5, 8.0])), spare_q=int(rng.integers(0, 3)),
             spare_kv=int(rng.integers(0, 3)), layout=str(rng.choice(["packed", "apart", "shared"])),
             scale=float(rng.choice([R.SCALE, -0.05, 0.2])))
    c.put().run().check()


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_query_magnitudes(kind):
    """Rows of very different sizes, and rows whose elements are."""
    c = Call([8], [200], 1, dtype=kind[0], kv=kind[1], causal=False)
    q = c.q.float()
    if kind[0] is BF:
        q[0] *= 1e-30
        q[1] *= 2.0 ** -100
    q[2] *= 30
    q[3, :, ::7] *= 100
    q[4] *= torch.exp(torch.linspace(-12, 1, 192))
    q[5] = 0
    q[6] = 0
    q[6, 0, 191] = 8
    c.q = q.to(kind[0])
    c.put().run().check()


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_growing_scores_and_long_tails(kind):
    """Scores that grow along the row (references move often), fall, and one large weight with a
    long tail of equal small ones that hold a fifth of the mass."""
    c = Call([2], [2000], 1, dtype=kind[0], kv=kind[1], causal=False, scale=1.0)
    ks = c.kv_scale or 1.0
    q, key = torch.zeros(2, 1, 192), torch.zeros(2000, 1, 192)
    q[0, 0, 0] = 1.0
    q[1, 0, 1] = 1.0
    key[:, 0, 0] = torch.linspace(-60, 60, 2000) / ks   # rises
    key[:, 0, 1] = torch.linspace(40, -40, 2000) / ks   # falls
    lim = 400.0 if kind[1] is E4 else 5e4
    c.q, c.key = q.to(kind[0]), key.clamp(-lim, lim).to(kind[1])
    c.put().run().check()
    key[:, 0, 0] = 0
    key[77, 0, 0] = float(np.log(4 * 1999)) / ks
    c.key = key.clamp(-lim, lim).to(kind[1])
    c.put().run().check()


NAN_ROW = {BF: 0x7FC0, HF: 0x7E00}


@pytest.mark.parametrize("kind", KINDS, ids=str)
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_bad_rows_stay_unseen(kind, bad):
    """Rows behind a sequence, and rows that come after a token, hold NaN or infinities: tokens
    that do not see them keep their bits."""
    lens = ([100, 200], [230, 200])
    clean = Call(*lens, 2, dtype=kind[0], kv=kind[1], spare_kv=140).put().run().got()
    c = Call(*lens, 2, dtype=kind[0], kv=kind[1], spare_kv=140)
    if c.kv is E4 and bad == "inf":
        pytest.skip("e4m3 has no infinity")
    val = float("nan") if bad == "nan" else float("inf")
    key, v = c.key.float(), c.v.float()
    for x in (key, v):
        x[430:] = val             # behind the last sequence
        x[230 + 90] = val         # seen from the second sequence's token 90 on
        x[230 + 199, :, 5] = val  # by its last token
        x[229] = val              # by the first sequence's last token
    c.key, c.v = (x.to(c.kv) if bad == "nan" else _with_inf(x, c.kv) for x in (key, v))
    out, lse, e = c.put().run().got()
    sees = np.zeros(300, bool)
    sees[99] = True
    sees[100 + 90:] = True
    assert np.array_equal(out[~sees], clean[0][~sees]) and np.array_equal(lse[~sees], clean[1][~sees])
    if bad == "nan":
        assert np.isnan(out[99]).all()
    assert e == 0


def _with_inf(x, dtype):
    y = x.clamp(-5e4, 5e4).to(dtype)
    if dtype is E5:
        y.view(torch.uint8)[torch.isinf(x)] = 0x7C
    else:
        y[torch.isinf(x)] = float("inf")
    return y


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("kv", [BF, E4])
def test_a_bad_query_row_stays_alone(bad, kv):
    good = Call([200], [200], 2, kv=kv).put().run().got()
    c = Call([200], [200], 2, kv=kv)
    c.q[130, 1, 100] = bad
    out, lse, _ = c.put().run().got()
    rest = np.ones((200, 2), bool)
    rest[130, 1] = False
    assert np.isnan(out[130, 1]).all()
    assert np.array_equal(out[rest], good[0][rest]) and np.array_equal(lse[rest], good[1][rest])


def test_rows_that_do_not_exist():
    """Key rows behind the arrays are left out and reported; tokens behind theirs are not touched."""
    c = Call([10, 20], [100, 60], 2)
    c.put()
    K = 130
    c.dk, c.dp, c.dv = c.dk[:K], c.dp[:K], c.dv[:K]
    c.run().check(err=8 // 2, limit=K)
    c = Call([10, 20], [100, 60], 2, spare_q=0)
    c.put()
    c.dq, c.out, c.lse = c.dq[:25], c.out[:25], c.lse[:25]
    c.q = c.q[:25]
    c.run()
    torch.cuda.synchronize()
    assert (c.out_full[25:, :, :128] == 7).all()
    r = c.expected()
    bo, bl = R.bounds(r, c.dtype, c.kv)
    assert (np.abs(R.f64(c.out.cpu()) - r.out) <= bo).all()


def test_unowned_tokens_and_empty_calls():
    c = Call([3, 4], [5, 6], 2, spare_q=5, spare_kv=5)
    c.cu_q = [2, 5, 9]
    c.put().run().check()
    c = Call([3, 4], [5, 6], 2)
    c.put()
    c.dq, c.out, c.lse = c.dq[:0], c.out[:0], c.lse[:0]
    c.run()
    torch.cuda.synchronize()
    assert (c.out_full[:, :, :128] == 7).all()
    c = Call([3, 4], [0, 0], 2)  # no key rows at all
    c.put().run().check()


def test_no_lse():
    c = Call([30], [30], 2).put()
    c.run(lse=None)
    torch.cuda.synchronize()
    assert (c.lse_full == 7).all()
    out = R.f64(c.out.cpu())
    assert np.array_equal(out, Call([30], [30], 2).put().run().got()[0])


def test_many_sequences():
    """More sequences than one block looks at in a round, most of them of a few tokens, some empty."""
    rng = np.random.default_rng(3)
    ql = [int(x) for x in rng.integers(0, 4, 700)]
    kl = [q + int(x) for q, x in zip(ql, rng.integers(0, 40, 700))]
    Call(ql, kl, 1).put().run().check()


def test_broadcast_heads():
    """All heads share one key and value row (head strides of 0)."""
    c = Call([50], [90], 4, 4)
    c.key = c.key[:, :1].expand(-1, 4, -1).contiguous()
    c.v = c.v[:, :1].expand(-1, 4, -1).contiguous()
    c.put()
    c.dk, c.dp, c.dv = (t[:, :1].expand(-1, 4, -1) for t in (c.dk, c.dp, c.dv))
    c.run().check()


def test_calls_repeat_to_the_bit_on_streams_and_in_graphs():
    c = Call([1, 140, 2], [3000, 300, 200], 4).put().run()
    first = c.got()
    for x in (c.out_full, c.lse_full):
        x.fill_(3.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    s.synchronize()
    again = c.got()
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])
    c.out_full.fill_(3.0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
        c.run()
    for _ in range(3):
        g.replay()
    again = c.got()
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_two_graphs_with_one_workspace():
    """Calls of different shapes captured apart on one workspace, replayed in turn."""
    a, b = Call([1], [4000], 2).put().run(), Call([90, 90], [700, 90], 2, seed=5).put().run()
    wa, wb = a.got(), b.got()
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    a.ws = b.ws = ws
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for g in graphs * 3:
        g.replay()
    for c, w in ((a, wa), (b, wb)):
        o = c.got()
        assert np.array_equal(o[0], w[0]) and np.array_equal(o[1], w[1])


def test_long_items_between_others():
    """Items of many key tiles beside short ones, several in a block's run: results by 64-bit
    arithmetic on the device, the same bits every time, and no wait that runs out."""
    lens = [1400, 30, 2048, 700, 257, 1111]
    c = Call(lens, lens, 8, 8).put()
    ref = []
    for s, n in enumerate(lens):
        rows = slice(c.cu_q[s], c.cu_q[s + 1])
        q, key, v = c.dq[rows].double(), torch.cat([c.dk[rows], c.dp[rows]], -1).double(), c.dv[rows].double()
        x = torch.einsum("the,khe->htk", q, key) * c.scale
        x.masked_fill_(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -np.inf)
        ref.append(torch.einsum("htk,khe->the", torch.softmax(x, -1), v))
    ref = torch.cat(ref)
    first = None
    for _ in range(60):
        c.run()
        out = c.out.clone()
        assert first is None or torch.equal(out, first)
        first = out
    assert int(c.err.item()) == 0
    # weights and the result round to bf16: 2^-8 of the row's magnitude each, and of the value
    mag = 2.0 ** -8 * (2 + 2.0 ** -6) * 4.5  # |v| stays below 4.5 in all but a few of 10^6 values
    assert c.dv.abs().max() < 6 and (first.double() - ref).abs().max() < mag * 6 / 4.5
    assert (first.double() - ref).norm() < 2.0 ** -8 * ref.norm()


@pytest.mark.parametrize("kind,heads,kv_heads", [((BF, E4), 6, 2), ((HF, E5), 5, 1), ((BF, E4), 40, 1), ((HF, HF), 6, 2)], ids=str)
def test_head_layouts_of_other_types(kind, heads, kv_heads):
    Call([33, 1, 60], [33, 200, 170], heads, kv_heads, *kind).put().run().check()


@pytest.mark.parametrize("seqs,heads,kv_heads,kv", [
    (150, 1, 1, 512), (150, 1, 1, 513), (151, 1, 1, 450), (4, 32, 32, 512), (4, 32, 32, 520), (1, 256, 1, 512),
    (1, 256, 2, 513), (150, 1, 1, 768), (150, 1, 1, 769), (151, 1, 1, 700), (1, 256, 1, 768), (1, 256, 2, 769)],
    ids=str)
def test_borders_of_whole_items(seqs, heads, kv_heads, kv):
    """Around the sizes from which items are cut: 768 key rows in all, an item per SM."""
    lens = [kv // seqs] * (seqs - 1) + [kv - kv // seqs * (seqs - 1)]
    Call([min(2, n) for n in lens], lens, heads, kv_heads, BF).put().run().check()


@pytest.mark.parametrize("kind", [(BF, BF), (HF, HF), (BF, E4)], ids=str)
@pytest.mark.parametrize("lens", [([300], [300]), ([300, 20], [1300, 400])], ids=str)
def test_rows_of_out_on_32_bytes(kind, lens):
    """out without gaps, which is written in wider stores; and the same bits with gaps."""
    c = Call(*lens, heads=4, dtype=kind[0], kv=kind[1]).put().run()
    first = c.got()
    T, H = c.out.shape[:2]
    out = torch.full((T, H, 128), 7.0, dtype=kind[0], device="cuda")
    ops.mla_prefill_attention(c.dq[:, :, :128], c.dq[:, :, 128:], c.dk, c.dp, c.dv, c.dcq, c.dck, out, c.ws,
                              softmax_scale=c.scale, kv_scale=c.ds)
    torch.cuda.synchronize()
    assert np.array_equal(R.f64(out.cpu()), first[0])


@pytest.mark.parametrize("kind", [(BF, BF), (HF, HF), (BF, E4)], ids=str)
@pytest.mark.parametrize("scale", [0.0, -R.SCALE, 1e-30])
def test_scales(kind, scale):
    Call([70, 200], [70, 330], heads=2, dtype=kind[0], kv=kind[1], scale=scale).put().run().check()


@pytest.mark.parametrize("which", ["heads", "tokens"])
@pytest.mark.parametrize("kind", [(BF, BF), (BF, E4)], ids=str)
def test_broadcast_queries(kind, which):
    """Queries whose heads, or tokens, are one row."""
    c = Call([70, 40], [70, 300], heads=4, dtype=kind[0], kv=kind[1])
    c.q = (c.q[:, :1].expand(-1, 4, -1) if which == "heads" else c.q[:1].expand(110, -1, -1)).clone()
    c.put()
    c.dq = c.dq[:, :1].expand(-1, 4, -1) if which == "heads" else c.dq[:1].expand(110, -1, -1)
    c.run().check()


def test_offsets_past_32_bits():
    """Rows 16 MiB apart in one buffer of 5 GB: queries, keys, values and results side by side."""
    c = Call([300], [310], heads=1).put()
    step, n = 1 << 23, 310
    big = torch.empty(n * step, dtype=BF, device="cuda")
    at = lambda off, w, rows: big.as_strided((rows, 1, w), (step, 192, 1), off)
    q, key, v, out = at(0, 192, 300), at(192, 192, n), at(384, 128, n), at(512, 128, 300)
    q.copy_(c.dq)
    key[:, :, :128].copy_(c.dk)
    key[:, :, 128:].copy_(c.dp)
    v.copy_(c.dv)
    ops.mla_prefill_attention(q[:, :, :128], q[:, :, 128:], key[:, :, :128], key[:, :, 128:], v, c.dcq, c.dck, out,
                              c.ws, softmax_scale=c.scale, lse=c.lse, err_word=c.err)
    c.out.copy_(out)
    c.check()


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, repeat what they give alone."""
    calls = [Call([700, 30], [900, 1500], 8, 2, seed=1).put(), Call([1, 300], [2000, 300], 4, 4, BF, E4, seed=2).put()]
    alone = [c.run().got()[0] for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    for c in calls:
        c.out.fill_(3.0)
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, streams):
            c.run(stream=s)
    for c, want in zip(calls, alone):
        assert np.array_equal(c.got()[0], want)


def test_device_refusals():
    c = Call([5], [5]).put()
    ws = c.ws
    c.ws = ws[:-16]
    with pytest.raises(ops.MlaError, match="workspace_bytes must be >="):
        c.run()
    c.ws = ws
    c.dv = c.dv.cpu()
    with pytest.raises(ops.MlaError, match="v must be device memory"):
        c.run()


@pytest.mark.parametrize("kind,stages", [((BF, BF), 6), ((HF, HF), 6), ((BF, E4), 4)], ids=str)
def test_waits_that_run_out_return_and_report(kind, stages):
    """With a 1 ms limit and a stage of the first CTA that never fills (a testing hook), its waits
    run out: the call returns and says so, the other CTAs' heads are as ever, and the next call is
    exact.  No fault is involved: only bounded waits that give up."""
    c = Call([2000], [2000], 8, dtype=kind[0], kv=kind[1]).put()
    good = c.run().got()[0]
    for stage in range(1, stages + 1):
        c.out.fill_(3.0)
        torch.cuda.synchronize()
        try:
            ops.mla_test_attention_timeout(1_000_000, stage)
            out, _, e = c.run().got()
        finally:
            ops.mla_test_attention_timeout()
        assert e == ops.MLA_ERRBIT_TIMEOUT
        assert np.array_equal(out[:, 2:], good[:, 2:]) and not np.array_equal(out[:, 0], good[:, 0])
        c.err.zero_()
        out, _, e = c.run().got()
        assert e == 0 and np.array_equal(out, good)


@pytest.mark.parametrize("kind", [(BF, BF), (HF, HF), (BF, E4)], ids=str)
def test_heads_outside_of_tokens(kind):
    """[head, token, element] arrays, seen as [token, head, element]: queries, keys, values, results."""
    c = Call([150, 40], [280, 300], 4, 2, *kind).put()
    swap = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)
    c.dq, c.dv = swap(c.dq), swap(c.dv)
    key = swap(torch.cat([c.dk.view(torch.uint8), c.dp.view(torch.uint8)], -1)).view(kind[1])
    c.dk, c.dp = key[:, :, :128], key[:, :, 128:]
    full = torch.full((4, 191, 136), 7.0, dtype=kind[0], device="cuda")
    c.out_full, c.out = full.transpose(0, 1), full.transpose(0, 1)[:190, :, :128]
    c.run().check()


def test_lists_that_are_not_whole():
    """Sequences without keys, without tokens, and with fewer keys than tokens, next to each other."""
    Call([0, 9, 0, 300, 2, 0, 70], [5, 0, 0, 200, 0, 900, 1], 3, 1).put().run().check()
    Call([9, 0, 0, 1], [0, 0, 70, 0], 2, 2, HF, E5, causal=False).put().run().check()


@pytest.mark.parametrize("kind,causal", [((HF, HF), True), ((BF, BF), False), ((BF, E4), True)], ids=str)
def test_many_calls_give_the_same_bits(kind, causal):
    """Items of one query tile between others of two, 4000 times: warps of a tile that has no rows in
    an item are held back by little, and must not take one phase of a barrier for another."""
    rng = np.random.default_rng(7)
    q = [int(x) for x in rng.choice([0, 1, 2, 60, 90, 262, 286, 346], 150)]
    c = Call(q, [x + int(rng.integers(0, 60)) for x in q], 6, 2, *kind, causal=causal).put().run()
    first, lse = c.out.clone(), c.lse.clone()
    differ = torch.zeros((), dtype=torch.bool, device="cuda")
    for _ in range(4000):
        c.run()
        differ |= (c.out.view(torch.int16) != first.view(torch.int16)).any() | (c.lse != lse).any()
    assert not differ.item() and c.err.item() == 0


@pytest.mark.parametrize("kind", KINDS, ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("kv_lens", [[70, 0, 200], [400, 0, 900]], ids=str)
def test_bad_queries_that_see_no_row(kind, bad, kv_lens):
    """A token that sees nothing has 0 and -infinity, whatever its query holds (a padded batch's
    rows): more tokens than rows, no rows at all, and those beside them as ever."""
    lens = [100, 30, 210] if kv_lens[0] == 70 else [430, 30, 905]
    none = np.zeros(sum(lens), bool)
    none[:30] = none[lens[0]:lens[0] + 30] = True
    none[lens[0] + 30:lens[0] + 30 + lens[2] - kv_lens[2]] = True
    good = Call(lens, kv_lens, 3, 1, *kind).put().run()
    good.check()
    want = good.got()
    c = Call(lens, kv_lens, 3, 1, *kind)
    c.q[torch.from_numpy(none)] = bad
    out, lse, e = c.put().run().got()
    assert (out[none] == 0).all() and np.isneginf(lse[none]).all() and e == 0
    assert np.array_equal(out, want[0]) and np.array_equal(lse, want[1])


def _same_bits(a, b):
    """Results of `got`, NaNs among them."""
    return all(np.array_equal(x, y, equal_nan=True) for x, y in zip(a, b))


@pytest.mark.parametrize("kind", KINDS, ids=str)
@pytest.mark.parametrize("ctx", [160, 900])
def test_a_large_key_moves_no_row_that_does_not_see_it(kind, ctx):
    """Tokens 25 to 63 see a key whose scores dwarf the others; the tokens before them, some of them
    rows of the same warp, keep every bit.  The key lies behind a tile of smaller ones (of the
    block's part of the sum, too, where that is cut), so its reader's reference has to move."""
    p = ctx + 25
    got = []
    for mul in (1.0, 20.0 if kind[1] not in R.FP8 else 10.0):
        c = Call([64], [ctx + 64], 4, dtype=kind[0], kv=kind[1])
        key = c.key.float()
        key[:p // 64 * 64] *= 0.5
        key[p] *= mul
        c.key = (key.clamp(-448, 448) if kind[1] is E4 else key).to(kind[1])
        c.put().run().check()
        got.append(c.got()[:2])
    assert _same_bits([x[:25] for x in got[0]], [x[:25] for x in got[1]])
    assert not np.array_equal(got[0][1][25:], got[1][1][25:])


@pytest.mark.parametrize("kind", KINDS, ids=str)
def test_queries_of_the_next_sequence_move_no_row(kind):
    """Tokens of the next sequence that share a warp's rows with this one's last tokens: whatever
    they ask, this sequence keeps every bit."""
    got = []
    for mul in (1.0, 40.0, float("nan")):
        c = Call([20, 200], [300, 300], 2, dtype=kind[0], kv=kind[1])
        key = c.key.float()
        key[:128] *= 0.5
        c.key = key.to(kind[1])
        c.q[20:] *= mul
        c.put().run()
        got.append(c.got()[:2])
    for other in got[1:]:
        assert _same_bits([x[:20] for x in got[0]], [x[:20] for x in other])


@pytest.mark.parametrize("kind", [(BF, BF), (HF, HF), (BF, E4)], ids=str)
@pytest.mark.parametrize("rows", [1, 2])
def test_heads_far_apart(kind, rows):
    """Heads 2^30 elements apart: the columns of three of them are more than 2^31, outside of the one
    row that there is, or (two rows) inside of rows that are farther apart still."""
    heads, step = 3, (1 << 30) + 64
    c = Call([5], [rows], heads, dtype=kind[0], kv=kind[1]).put()
    big = torch.empty((rows - 1) * (3 * step) + 2 * step + 128, dtype=kind[1], device="cuda")
    far = big.as_strided((rows, heads, 128), (3 * step, step, 1))
    far.view(torch.uint8).copy_(c.dk.contiguous().view(torch.uint8))
    c.dk = far
    c.run().check()


@pytest.mark.parametrize("kind,stages", [((BF, BF), 6), ((HF, E5), 4)], ids=str)
def test_waits_that_run_out_with_queries_on_their_way(kind, stages):
    """As above, with many short items, so that query boxes of both tiles come again and again (also
    of tiles without rows): the call ends, says so, and the next one, launched right behind it, is
    exact."""
    lens = [130, 20, 300, 129, 70, 256] * 40
    c = Call(lens, lens, 4, 2, *kind).put()
    good = c.run().got()[0]
    for stage in range(1, stages + 1):
        c.out.fill_(3.0)
        torch.cuda.synchronize()
        try:
            ops.mla_test_attention_timeout(1_000_000, stage)
            c.run()
        finally:
            ops.mla_test_attention_timeout()
        first = c.out.clone()
        c.run()
        out, _, e = c.got()
        assert e == ops.MLA_ERRBIT_TIMEOUT and np.array_equal(out, good)
        assert not np.array_equal(R.f64(first.cpu())[:130, :2], good[:130, :2])
        c.err.zero_()


@pytest.mark.parametrize("seed", range(12))
def test_many_calls_of_many_shapes_give_the_same_bits(seed):
    """12 x 10 random batches, 400 calls of each: what a call gives does not depend on when its warps
    come by."""
    rng = np.random.default_rng(900 + seed)
    for i in range(10):
        n, G = int(rng.choice([1, 3, 12, 60, 150])), int(rng.choice([1, 2, 4]))
        H = G * int(rng.choice([1, 2, 3, 8]))
        most = max(2, min(1200, 40000 // (n * H)))
        ql = [int(rng.choice([0, 1, 2, 60, 127, 130, int(rng.integers(1, most + 1))])) for _ in range(n)]
        ql[0] = max(1, ql[0])
        kind = KINDS[int(rng.integers(0, len(KINDS)))]
        c = Call(ql, [x + int(rng.choice([0, 1, 30, 64, 700 // n])) for x in ql], H, G, *kind, seed=i,
                 causal=bool(rng.integers(0, 2))).put().run()
        out, lse = c.out.clone(), c.lse.clone()
        differ = torch.zeros((), dtype=torch.bool, device="cuda")
        for _ in range(400):
            c.run()
            differ |= (c.out.view(torch.int16) != out.view(torch.int16)).any() | (c.lse != lse).any()
        assert not differ.item() and c.err.item() == 0, (i, ql, H, G, kind)


@pytest.mark.parametrize("kind", [(BF, BF), (HF, HF), (BF, E4), (HF, E5)], ids=str)
def test_batches_whose_units_are_counted_in_64_bits(kind):
    """4096 sequences, nearly all empty: by an estimate from their number the units could pass 32
    bits.  The same four sequences alone stay below it; nothing else differs, so the bits agree, and
    tokens of each agree with 64-bit arithmetic."""
    lens, kvs, at = [1300, 1, 499, 200], [9000, 4000, 5000, 2000], [0, 17, 2000, 4095]
    H, G = 256, 64
    T, K = sum(lens), sum(kvs)
    q = R.values((T, H, 192), kind[0], 1, 1.5).cuda()
    mul = 30.0 if kind[1] in R.FP8 else 1.0
    key, v = R.values((K, 1, 192), kind[1], 2, mul).cuda(), R.values((K, 1, 128), kind[1], 3, mul).cuda()
    key, v = key.expand(-1, G, -1), v.expand(-1, G, -1)
    ks = torch.tensor([0.03], device="cuda") if kind[1] in R.FP8 else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    got = []
    for n in (4, 4096):
        ql, kl = np.zeros(n, int), np.zeros(n, int)
        where = range(4) if n == 4 else at
        for s, a, b in zip(where, lens, kvs):
            ql[s], kl[s] = a, b
        out, lse = torch.full((T, H, 128), 7.0, dtype=kind[0], device="cuda"), torch.full((T, H), 7.0, device="cuda")
        ws = torch.full((ops.mla_prefill_attention_workspace(T, H, G, n),), 0xFF, dtype=torch.uint8, device="cuda")
        ops.mla_prefill_attention(q[:, :, :128], q[:, :, 128:], key[:, :, :128], key[:, :, 128:], v, i32(cu_of(ql)),
                                  i32(cu_of(kl)), out, ws, softmax_scale=R.SCALE, kv_scale=ks, lse=lse, err_word=err)
        torch.cuda.synchronize()
        got.append((out, lse))
    assert torch.equal(got[0][0].view(torch.int16), got[1][0].view(torch.int16)) and torch.equal(got[0][1], got[1][1])
    assert err.item() == 0
    c = 1.0 if ks is None else float(np.float32(0.03))
    cq, ck = cu_of(lens), cu_of(kvs)
    for s in range(4):
        for t in {0, lens[s] // 2, lens[s] - 1}:
            m = kvs[s] - lens[s] + 1 + t
            rows = slice(ck[s], ck[s] + m)
            r = R.attend(R.f64(q[cq[s] + t:cq[s] + t + 1, ::17].cpu()), c * R.f64(key[rows, :1].cpu()),
                         c * R.f64(v[rows, :1].cpu()), [0, 1], [0, m], R.SCALE, False)
            bo, bl = R.bounds(r, kind[0], kind[1])
            assert (np.abs(R.f64(got[1][0][cq[s] + t:cq[s] + t + 1, ::17].cpu()) - r.out) <= bo).all()
            assert (np.abs(R.f64(got[1][1][cq[s] + t:cq[s] + t + 1, ::17].cpu()) - r.lse) <= bl).all()
