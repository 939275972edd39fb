"""GPU parity of mla_merge_attn_states (float64 reference, derived bounds) and
mla_cache_copy_blocks (byte-exact), and a run of the serving operators together:
insert, fork, attention over the shared prefix and over each suffix, merge."""
import numpy as np
import pytest
import torch

import devutil as D
import refattn as R
from pack_mla_cache_gb300 import ops
from pack_mla_cache_gb300 import workloads as W

pytestmark = pytest.mark.gpu
TYPES = {"bf16": (torch.bfloat16, R.BF16_HALF), "fp16": (torch.float16, R.FP16_HALF),
         "fp32": (torch.float32, R.FP32_HALF)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pack_mla_cache_gb300 import build
    build.build()
    ops.lib()


# ------------------------------------------------------------------------ merge
def merge_case(P, T, H, Dm, kind, seed=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    parts = torch.randn(P, T, H, Dm, generator=g).to(TYPES[kind][0])
    lse = spread * torch.randn(P, T, H, generator=g) + 5
    lse[torch.rand(P, T, H, generator=g) < 0.2] = -np.inf
    parts[lse == -np.inf] = float("nan")  # a part that saw nothing has no influence
    return parts, lse


def merge_check(orc, out, lo, parts, lse, kind):
    ro, rl = orc.merge_attn_states(parts.double().numpy(), lse.double().numpy())
    P = parts.shape[0]
    # a weight exp(lse_i - m): the difference is rounded once (2^-24 of up to |lse_i - m|), expf is
    # within 2 units; P additions and multiplications of half a unit each, the reciprocal and the
    # product; then one rounding to the type
    finite = torch.where(torch.isfinite(lse), lse, torch.zeros(()))
    span = float(2 * finite.abs().max())
    rel = (span + 4 + 2 * P + 4) * 2 * R.FP32_HALF
    with np.errstate(invalid="ignore"):
        mag = np.nan_to_num(np.abs(parts.double().numpy())).max(0)
    tiny = 2.0 ** -25 if kind == "fp16" else 1e-37  # half the smallest subnormal
    bound = rel * mag + TYPES[kind][1] * (np.abs(ro) + rel * mag) + tiny
    out = out.double().cpu().numpy()
    assert (np.abs(out - ro) <= bound).all(), (np.abs(out - ro) / bound).max()
    none = np.isneginf(rl)
    assert (out[none] == 0).all()
    if lo is not None:
        lo = lo.double().cpu().numpy()
        assert np.isneginf(lo[none]).all()
        assert (np.abs(lo[~none] - rl[~none]) <= rel + 4 * R.FP32_HALF * np.abs(rl[~none])).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("P,T,H,Dm", [(1, 1, 1, 8), (2, 3, 16, 512), (3, 65, 3, 128), (5, 17, 2, 192),
                                      (16, 9, 16, 128), (37, 5, 3, 24), (2, 700, 16, 512)])
def test_merge_parity(orc, kind, P, T, H, Dm):
    parts, lse = merge_case(P, T, H, Dm, kind)
    out = torch.full((T + 1, H, Dm), 7.0, dtype=parts.dtype, device="cuda")
    lo = torch.full((T + 1, H), 7.0, device="cuda")
    ops.mla_merge_attn_states(parts.cuda(), lse.cuda(), out[:T], lse_out=lo[:T])
    torch.cuda.synchronize()
    merge_check(orc, out[:T], lo[:T], parts, lse, kind)
    assert (out[T] == 7).all() and (lo[T] == 7).all()


def test_merge_strides(orc):
    """Head-major parts and log-sum-exps, padded rows, a strided output, no lse_out."""
    P, T, H, Dm = 3, 20, 6, 64
    parts, lse = merge_case(P, T, H, Dm, "bf16")
    p = torch.zeros(P, H, T, Dm + 8, dtype=torch.bfloat16, device="cuda")
    p[..., :Dm] = parts.transpose(1, 2)
    le = lse.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    out = torch.full((H, T, Dm + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.mla_merge_attn_states(p[..., :Dm].transpose(1, 2), le, out[..., :Dm].transpose(0, 1))
    torch.cuda.synchronize()
    merge_check(orc, out[..., :Dm].transpose(0, 1), None, parts, lse, "bf16")
    assert (out[..., Dm:] == 7).all()


@pytest.mark.parametrize("spread", [1e-3, 60.0])
def test_merge_spread_of_lse(orc, spread):
    parts, lse = merge_case(4, 50, 4, 128, "fp32", spread=spread)
    out, lo = torch.empty(50, 4, 128, device="cuda"), torch.empty(50, 4, device="cuda")
    ops.mla_merge_attn_states(parts.cuda(), lse.cuda(), out, lse_out=lo)
    torch.cuda.synchronize()
    merge_check(orc, out, lo, parts, lse, "fp32")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_merge_of_a_bad_lse_is_nan(bad):
    parts, lse = torch.ones(2, 2, 1, 8, device="cuda"), torch.zeros(2, 2, 1, device="cuda")
    lse[1, 0] = bad
    out, lo = torch.empty(2, 1, 8, device="cuda"), torch.empty(2, 1, device="cuda")
    ops.mla_merge_attn_states(parts, lse, out, lse_out=lo)
    assert out[0].isnan().all() and lo[0].isnan().all()
    assert (out[1] == 1).all() and lo[1].isfinite().all()


def test_merge_of_more_tokens_than_one_launch_takes():
    """2^31 - 1 tokens that share one row (strides of 0) of 16 bytes: two launches."""
    parts = torch.tensor([[1.0] * 8, [3.0] * 8], dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(2, device="cuda")
    out, lo = torch.zeros(8, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, device="cuda")
    T = 2 ** 31 - 1
    ops.mla_merge_attn_states(parts.as_strided((2, T, 1, 8), (8, 0, 0, 1)),
                              lse.as_strided((2, T, 1), (1, 0, 0)),
                              out.as_strided((T, 1, 8), (0, 0, 1)),
                              lse_out=lo.as_strided((T, 1), (0, 0)))
    torch.cuda.synchronize()
    assert (out == 2).all()
    assert abs(float(lo) - np.log(2)) < 4 * R.FP32_HALF


def test_merge_refuses_host_memory():
    p = torch.zeros(2, 1, 1, 8, device="cuda")
    with pytest.raises(ops.MlaError, match="lse must be device memory"):
        ops.mla_merge_attn_states(p, torch.zeros(2, 1, 1), torch.zeros(1, 1, 8, device="cuda"))


# ------------------------------------------------------------------ block copies
def copy_both(orc, L, nb, bs, bst, es, ed, fmt, src, dst, rows, seed=0, want_err=0, ptr_fix=None):
    rng = np.random.default_rng(seed)
    esz = 2 if fmt == 0 else 1
    host = [rng.integers(0, 256, nb * bst * esz).astype(np.uint8) for _ in range(L)]
    bufs = [D.Guarded(nb * bst * esz) for _ in range(L)]
    for b, h in zip(bufs, host):
        b.t.copy_(torch.from_numpy(h))
    ptrs = torch.tensor([b.ptr() for b in bufs], dtype=torch.int64, device="cuda")
    skip = []
    if ptr_fix:
        skip = ptr_fix(ptrs)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda v: None if v is None else np.asarray(v, np.int32)
    up = lambda v: None if v is None else D.dev(i32(v))
    ops.mla_cache_copy_blocks(ptrs, fmt, nb, bs, bst, es, ed, up(src), up(dst), row_counts=up(rows),
                              err_word=err)
    torch.cuda.synchronize()
    orc.copy_blocks([h for i, h in enumerate(host) if i not in skip], esz, nb, bs, bst, es, ed,
                    i32(src), i32(dst), i32(rows))
    for b, h in zip(bufs, host):
        np.testing.assert_array_equal(b.host(), h)
        assert b.guards_intact()
    assert int(err.item()) == want_err


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("bs,pad_e,pad_b", [(64, 0, 0), (16, 0, 0), (1, 0, 0), (48, 16, 32), (7, 32, 0)])
def test_copy_fork_clear(orc, fmt, bs, pad_e, pad_b):
    es = 576 + pad_e
    src = [3, 3, -1, 1, 2, 9, 4, 0]
    dst = [15, 6, 7, -1, 10, 9, 12, 13]
    rows = [bs, (bs + 1) // 2, bs, bs, 0, bs, 1, max(1, bs - 1)]
    copy_both(orc, 5, 17, bs, bs * es + pad_b, es, 576, fmt, src, dst, rows)
    copy_both(orc, 3, 17, bs, bs * es + pad_b, es, 576, fmt, src, dst, None)


@pytest.mark.parametrize("dim", [16, 512, 1024])
def test_copy_other_entry_sizes(orc, dim):
    copy_both(orc, 2, 6, 5, 5 * 1040, 1040, dim, 1, [0, 1], [2, 3], [5, 2])


def test_copy_bad_ids_and_counts(orc):
    copy_both(orc, 2, 8, 16, 16 * 576, 576, 576, 1, [0, 8, 1, -2, 2, 3], [4, 5, 8, 6, -2, 7],
              [16, 1, 1, 1, 1, 17], want_err=ops.MLA_ERRBIT_BLOCK_OOB)
    copy_both(orc, 2, 8, 16, 16 * 576, 576, 576, 1, [0], [4], [-1],
              want_err=ops.MLA_ERRBIT_BLOCK_OOB)


def test_copy_skips_bad_layers(orc):
    def fix(ptrs):
        ptrs[1] = 0
        ptrs[2] += 8
        return [1, 2]
    copy_both(orc, 4, 8, 16, 16 * 576, 576, 576, 1, [0, 1], [4, 5], None,
              want_err=ops.MLA_ERRBIT_MISALIGNED, ptr_fix=fix)


def test_copy_many(orc):
    rng = np.random.default_rng(4)
    ids = rng.permutation(600)
    rows = rng.integers(0, 65, 300)
    copy_both(orc, 6, 600, 64, 64 * 576, 576, 576, 1, ids[:300], ids[300:], rows)


def test_copy_offsets_past_32_bits():
    n = (1 << 32) // (64 * 1152) + 3
    c = torch.zeros(n, 64, 576, dtype=torch.int16, device="cuda")
    c[1] = torch.arange(64 * 576, device="cuda").view(64, 576).to(torch.int16)
    ptrs = torch.tensor([c.data_ptr()], dtype=torch.int64, device="cuda")
    i = lambda v: torch.tensor([v], dtype=torch.int32, device="cuda")
    ops.mla_cache_copy_blocks(ptrs, 0, n, 64, 64 * 576, 576, 576, i(1), i(n - 1))
    ops.mla_cache_copy_blocks(ptrs, 0, n, 64, 64 * 576, 576, 576, i(n - 1), i(n - 3))
    torch.cuda.synchronize()
    assert torch.equal(c[n - 1], c[1]) and torch.equal(c[n - 3], c[1]) and (c[n - 2] == 0).all()


def test_copy_captured():
    c = torch.arange(8 * 16 * 576, device="cuda").remainder(251).to(torch.uint8).view(8, 16, 576)
    ptrs = torch.tensor([c.data_ptr()], dtype=torch.int64, device="cuda")
    src, dst = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, -1], [5, -1]))
    g = torch.cuda.CUDAGraph()
    call = lambda: ops.mla_cache_copy_blocks(ptrs, 1, 8, 16, 16 * 576, 576, 576, src, dst)
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call()
    dst.copy_(torch.tensor([6, 7], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c[6], c[0]) and (c[7] == 0).all()


# ------------------------------------------------------------------- all together
@pytest.mark.parametrize("fmt", [0, 1])
def test_insert_fork_attend_merge(fmt):
    """A prompt of 150 rows is inserted in two layers and forked into three
    samples (whole pages shared, the part-filled one copied with its row count);
    each sample inserts two rows of its own and attends with two new tokens.
    Attention over each sample's own block table equals the merge of attention
    over the shared pages (all samples' tokens as one sequence, not causal) with
    attention over each sample's own pages."""
    bs, prompt, samples, new, H, L = 64, 150, 3, 2, 16, 2
    nb, shared = 16, prompt // bs
    rng = np.random.default_rng(8)
    esz = 2 if fmt == 0 else 1
    caches = [torch.zeros(nb * bs * 576 * esz, dtype=torch.uint8, device="cuda") for _ in range(L)]
    ptrs = torch.tensor([c.data_ptr() for c in caches], dtype=torch.int64, device="cuda")
    scales = None if fmt == 0 else torch.tensor([0.011, 0.017], device="cuda")
    tail = prompt - shared * bs

    def insert(rows, slots):
        x = D.dev_bf16(R.orc.bf16_from_f32_array(rows.astype(np.float32)))
        ops.mla_cache_insert_grouped(x[..., :512], x[..., 512:], D.dev(np.asarray(slots, np.int64)),
                                     ptrs, scales, fmt, nb, bs, bs * 576, 576)

    prompt_pages, own_pages = [4, 9, 2], [[2], [11], [7]]
    insert(rng.standard_normal((L, prompt, 576)),
           [prompt_pages[p // bs] * bs + p % bs for p in range(prompt)])
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    ops.mla_cache_copy_blocks(ptrs, fmt, nb, bs, bs * 576, 576, 576, i32([2, 2]), i32([11, 7]),
                              row_counts=i32([tail, tail]))
    insert(rng.standard_normal((L, samples * new, 576)),
           [own_pages[s][0] * bs + tail + j for s in range(samples) for j in range(new)])
    T = samples * new
    q = D.dev_bf16(R.queries(T, H))
    cu = i32([0, 2, 4, 6])
    ws = torch.empty(ops.mla_latent_attention_workspace(T, H, samples), dtype=torch.uint8, device="cuda")
    for layer in range(L):
        ks = None if fmt == 0 else scales[layer:layer + 1]

        def attend(table, cu_q, lens, causal, out, lse):
            ops.mla_latent_attention(q[:, :, :512], q[:, :, 512:], caches[layer], fmt, nb, bs,
                                     bs * 576, 576, i32(table), cu_q, i32(lens), out, ws,
                                     softmax_scale=R.SCALE, k_scale=ks, causal=causal, lse=lse)

        whole, lse_w = torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, device="cuda")
        attend([[4, 9, p[0]] for p in own_pages], cu, [prompt + new] * samples, True, whole, lse_w)
        parts = torch.empty(2, T, H, 512, dtype=torch.bfloat16, device="cuda")
        lses = torch.empty(2, T, H, device="cuda")
        attend([[4, 9]], i32([0, T]), [shared * bs], False, parts[0], lses[0])
        attend(own_pages, cu, [tail + new] * samples, True, parts[1], lses[1])
        out, lse = torch.empty_like(whole), torch.empty_like(lse_w)
        ops.mla_merge_attn_states(parts, lses, out, lse_out=lse)
        torch.cuda.synchronize()
        # the whole against the definition on the rows that the caches really hold
        raw = caches[layer].cpu().numpy()
        table = np.array([[4, 9, p[0]] for p in own_pages], np.int32)
        pg = R.Paged(raw.view(np.uint16) if fmt == 0 else raw, fmt, nb, bs, bs * 576, 576, table,
                     None if fmt == 0 else float(scales[layer]))
        qh = D.host_u16(q)
        kv = [prompt + new] * samples
        r = R.attention(pg, qh, [0, 2, 4, 6], kv)
        ro, rl, mag = r.out, r.lse, r.mag
        bo, bl = R.attention_bounds(r)
        f = lambda t: t.double().cpu().numpy()
        assert (np.abs(f(whole) - ro) <= bo).all() and (np.abs(f(lse_w) - rl) <= bl).all()
        # a part is within the same bounds of its own result, whose magnitudes are at most the rows';
        # the weighted sum of the parts' errors and one more rounding
        part_mag = np.abs(f(parts)).max(0) + mag
        bm = bo + 2 * (R.BF16_HALF + 2 * bl[..., None]) * part_mag * 2
        assert (np.abs(f(out) - ro) <= bm).all() and (np.abs(f(lse) - rl) <= 2 * bl).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("P,Dm", [(2, 64), (7, 24), (1024, 8)])
def test_merge_of_the_largest_values_stays_finite(kind, P, Dm):
    """The join of equal rows is the row, also near the type's largest value (half a step of
    the type, and the weights' own rounding: 1024 additions of half a unit at most)."""
    dt = TYPES[kind][0]
    top = torch.finfo(dt).max * 0.99
    parts = torch.full((P, 3, 2, Dm), top).to(dt).cuda()
    lse = torch.zeros(P, 3, 2, device="cuda")
    out, lo = torch.zeros(3, 2, Dm, dtype=dt, device="cuda"), torch.zeros(3, 2, device="cuda")
    ops.mla_merge_attn_states(parts, lse, out, lse_out=lo)
    want = float(parts[0, 0, 0, 0])
    rel = TYPES[kind][1] + 2 * (P + 8) * R.FP32_HALF
    assert (out.double() - want).abs().max().item() <= rel * want
    assert (lo.double() - np.log(P)).abs().max().item() <= 8 * R.FP32_HALF * (1 + np.log(P))


def test_copies_of_no_rows_are_padding(orc):
    """A count of 0 is padding whatever the ids are, next to copies that are not."""
    copy_both(orc, 2, 8, 16, 16 * 576, 576, 576, 1, [99, 0, -9, 0, 1], [1, 99, -9, 5, 6],
              [0, 0, 0, 16, 3])


def test_copies_onto_themselves_are_checked_first(orc):
    copy_both(orc, 2, 8, 16, 16 * 576, 576, 576, 1, [3, 4], [3, 4], [16, 2])
    copy_both(orc, 2, 8, 16, 16 * 576, 576, 576, 1, [8, 0], [8, 5], [16, 2],
              want_err=ops.MLA_ERRBIT_BLOCK_OOB)
