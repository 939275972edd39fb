"""The workspace of mla_latent_attention: as large as the call's query tile needs, and not
written behind its end by a call that splits every query tile over the SMs."""
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


def test_small_calls_need_less():
    n = {rows: ops.mla_latent_attention_workspace(1, rows, 1) for rows in (1, 16, 17, 32, 33, 128)}
    assert n[1] == n[16] < n[17] == n[32] < n[33] == n[128]
    # any number of sequences: a call of fewer has more rows in each
    assert ops.mla_latent_attention_workspace(64, 16, 64) == n[128]
    assert ops.mla_latent_attention_workspace(2 ** 31 - 1, 1, 4096) == n[128]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("tokens,heads,seqs", [(1, 16, 1), (1, 32, 1), (2, 16, 1), (2, 16, 2), (3, 32, 3),
                                               (1, 64, 1), (1, 128, 1)])
def test_nothing_is_written_behind_the_end(fmt, tokens, heads, seqs):
    kv = [5000] * seqs
    pg = R.paged([5000], fmt, 64, seed=7)
    q = D.dev_bf16(R.queries(tokens, heads))
    cache = D.dev_bf16(pg.cache) if fmt == 0 else D.dev(pg.cache)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table = i32(pg.table.tolist() * seqs)
    ks = None if fmt == 0 else torch.tensor([pg.k_scale], device="cuda")
    per = tokens // seqs
    need = ops.mla_latent_attention_workspace(tokens, heads, seqs)

    def run(ws):
        out = torch.empty(tokens, heads, 512, dtype=torch.bfloat16, device="cuda")
        ops.mla_latent_attention(q[:, :, :512], q[:, :, 512:], cache, fmt, pg.num_blocks, pg.block,
                                 pg.block_stride, pg.entry_stride, table,
                                 i32([per * i for i in range(seqs + 1)]), i32(kv), out, ws,
                                 softmax_scale=R.SCALE, k_scale=ks)
        torch.cuda.synchronize()
        return out

    whole = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    out = run(whole[:need])
    assert (whole[need:] == 0xA5).all()
    assert torch.equal(out, run(torch.empty(4 * need, dtype=torch.uint8, device="cuda")))
    with pytest.raises(ops.MlaError, match="workspace_bytes"):
        run(whole[:need - 1])
