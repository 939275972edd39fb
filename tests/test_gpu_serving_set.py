"""The serving operators one behind the other, as a server calls them: new tokens over a cached
context in chunks (pack, attention of each chunk, attention of the new tokens among themselves,
join), and the verification of drafted trees (attention, accepted rows moved, decode over them)."""
import numpy as np
import pytest
import torch

import devutil as D
import refattn as A
import refprefill as R
from pack_mla_cache_gb300 import ops

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pack_mla_cache_gb300 import build
    build.build()
    ops.lib()


def cu_of(lens):
    return [0] + [int(x) for x in np.cumsum(lens)]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fmt,graph", [(0, False), (1, False), (1, True)])
def test_new_tokens_over_a_cached_context(fmt, graph):
    """Two chunks of the context and the new tokens joined, against one attention over all.  A part
    is within its own bound; the join weighs parts by exp(lse_i - lse), off by a factor of twice the
    largest error of an lse, and adds fp32 roundings and one to bf16 (2^-8)."""
    H, new, ctx, chunk = 4, [70, 1, 33, 200], [300, 129, 0, 64], 160
    T, scale = sum(new), 0.03
    pg = A.paged(ctx, fmt, 16, seed=5, k_scale=scale)
    cache = D.dev_bf16(pg.cache) if fmt == 0 else D.dev(pg.cache)
    q = R.values((T, H, 192), BF, 1, 1.5).cuda()
    own = R.values((T, H, 256), BF, 2).cuda()  # the projection of the new tokens: keys, values
    own_pe = R.values((T, 64), BF, 3).cuda()
    cu_q = i32(cu_of(new))
    kd = BF if fmt == 0 else E4
    ds = None if fmt == 0 else torch.tensor([scale], device="cuda")
    chunks = []
    for c in range(2):
        lens = [max(0, min(chunk, n - c * chunk)) for n in ctx]
        up = R.values((max(1, sum(lens)), H, 256), BF, 7 + c).cuda()[:sum(lens)]
        chunks.append((lens, up, i32(cu_of(lens)), i32([c * chunk] * len(ctx)),
                       torch.zeros((sum(lens), H, 192), dtype=kd, device="cuda"),
                       torch.zeros((sum(lens), H, 128), dtype=kd, device="cuda")))
    parts = torch.full((3, T, H, 128), 7.0, dtype=BF, device="cuda")
    lses = torch.full((3, T, H), 7.0, device="cuda")
    out = torch.full((T, H, 128), 7.0, dtype=BF, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    ws = torch.empty(ops.mla_prefill_attention_workspace(T, H, H, len(new)), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = D.dev(pg.table)

    def step():
        for c, (lens, up, cu, starts, key, v) in enumerate(chunks):
            ops.mla_context_kv_pack_paged(up[:, :, :128], up[:, :, 128:], cache, fmt, pg.num_blocks, pg.block,
                                          pg.block_stride, pg.entry_stride, table, cu, starts, key, v, fmt,
                                          out_scale=ds, err_word=err)
            ops.mla_prefill_attention(q[:, :, :128], q[:, :, 128:], key[:, :, :128], key[:, :, 128:], v, cu_q, cu,
                                      parts[c], ws, softmax_scale=R.SCALE, causal=False, kv_scale=ds, lse=lses[c],
                                      err_word=err)
        ops.mla_prefill_attention(q[:, :, :128], q[:, :, 128:], own[:, :, :128], own_pe, own[:, :, 128:], cu_q, cu_q,
                                  parts[2], ws, softmax_scale=R.SCALE, lse=lses[2], err_word=err)
        ops.mla_merge_attn_states(parts, lses, out, lse_out=lse)

    step()
    if graph:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        out.fill_(3.0)
        for _ in range(2):
            g.replay()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    f, q64, s = (lambda t: R.f64(t.cpu())), R.f64(q.cpu()), scale if fmt else 1.0
    own_key = np.concatenate([f(own)[:, :, :128], np.repeat(f(own_pe)[:, None], H, 1)], -1)
    rs = [R.attend(q64, f(key) * s, f(v) * s, cu_of(new), cu_of(lens), R.SCALE, False)
          for lens, _, _, _, key, v in chunks]
    rs.append(R.attend(q64, own_key, f(own)[:, :, 128:], cu_of(new), cu_of(new), R.SCALE, True))
    whole = np.logaddexp.reduce([r.lse for r in rs], 0)
    w = [np.exp(r.lse - whole)[..., None] for r in rs]
    want = sum(a * r.out for a, r in zip(w, rs))
    bounds = [R.bounds(r, BF, k) for r, k in zip(rs, (kd, kd, BF))]
    worst = max(np.nanmax(np.where(np.isneginf(r.lse), 0, bl)) for r, (_, bl) in zip(rs, bounds))
    room = sum(a * (bo + np.abs(r.out) * (2 * worst + 2.0 ** -20)) for a, r, (bo, _) in zip(w, rs, bounds))
    room = room + 2.0 ** -8 * np.abs(want)
    assert (np.abs(f(out) - want) <= room).all()
    assert (np.abs(f(lse) - whole) <= worst + 2.0 ** -20 * (1 + np.abs(whole))).all()


@pytest.mark.parametrize("fmt", [0, 1])
def test_a_drafted_tree_verified_accepted_and_decoded(fmt):
    """The row of an accepted node, and a decode with its query after its branch was moved to the
    front, are the same attention over the same rows: both within the bound."""
    n, ctx, H = [8, 5, 16], [100, 40, 513], 16
    kv = [a + b for a, b in zip(n, ctx)]
    pg = A.paged(kv, fmt, 16, seed=9)
    q, masks = A.queries(sum(n), H), R.tree_masks(n, 11)
    dq = D.dev_bf16(q)
    cache = D.dev_bf16(pg.cache) if fmt == 0 else D.dev(pg.cache)
    ks = None if pg.k_scale is None else torch.tensor([pg.k_scale], device="cuda")
    table, cu = D.dev(pg.table), cu_of(n)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    nodes = [cu[s] + n[s] - 1 for s in range(3)]           # the accepted branches' last nodes
    branch = [np.flatnonzero(masks[t]) for t in nodes]     # and their drafted tokens, in order
    lists = torch.zeros((3, 16), dtype=torch.int32)
    for s, b in enumerate(branch):
        lists[s, :len(b)] = torch.from_numpy(b)

    def attention(tree, q, cu, kv, extra):
        T = q.shape[0]
        out, lse = torch.full((T, H, 512), 7.0, dtype=BF, device="cuda"), torch.full((T, H), 7.0, device="cuda")
        ws = torch.empty(ops.mla_latent_attention_workspace(T, H, 3), dtype=torch.uint8, device="cuda")
        f = ops.mla_latent_tree_attention if tree else ops.mla_latent_attention
        f(q[:, :, :512], q[:, :, 512:576], cache, fmt, pg.num_blocks, pg.block, pg.block_stride, pg.entry_stride,
          table, i32(cu), i32(kv), *extra, out, ws, softmax_scale=A.SCALE, k_scale=ks, lse=lse, err_word=err)
        return out, lse

    words = D.dev(R.words_of(masks))
    out, lse = attention(True, dq, cu, kv, [words])
    ptrs = torch.tensor([cache.data_ptr()], dtype=torch.int64, device="cuda")
    ops.mla_cache_compact_rows(ptrs, fmt, pg.num_blocks, pg.block, pg.block_stride, pg.entry_stride, 576, table,
                               i32(ctx), lists.cuda(), i32([len(b) for b in branch]), err_word=err)
    kept = [c + len(b) for c, b in zip(ctx, branch)]
    out2, lse2 = attention(False, dq[nodes].contiguous(), [0, 1, 2, 3], kept, [])
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    pg.cache = cache.cpu().view(torch.uint16 if fmt == 0 else torch.uint8).numpy()
    r = A.attention(pg, q[nodes], [0, 1, 2, 3], kept)
    bo, bl = A.attention_bounds(r)
    for o, l in ((out[nodes], lse[nodes]), (out2, lse2)):
        assert (np.abs(R.f64(o.cpu()) - r.out) <= bo).all()
        assert (np.abs(R.f64(l.cpu()) - r.lse) <= bl).all()
