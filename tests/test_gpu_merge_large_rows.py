"""mla_merge_attn_states on rows of 4 GiB: a thread's two chunks of such a row are 2^31 bytes
apart."""
import pytest
import torch

from pack_mla_cache_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pack_mla_cache_gb300 import build
    build.build()
    ops.lib()


@pytest.mark.parametrize("dtype,dim", [(torch.float32, 1 << 30), (torch.bfloat16, (1 << 31) - 16)])
def test_merge_of_rows_of_4_gib(dtype, dim):
    """A row joined with itself is the row: two equal weights, exact in fp32."""
    row = torch.empty(dim, dtype=dtype, device="cuda")
    for i in range(0, dim, 1 << 28):  # (in pieces: no second row of int64)
        n = min(1 << 28, dim - i)
        row[i:i + n] = torch.arange(n, device="cuda", dtype=torch.int32).remainder(251) + i // (1 << 28)
    out = torch.zeros(1, 1, dim, dtype=dtype, device="cuda")
    lo = torch.zeros(1, 1, device="cuda")
    ops.mla_merge_attn_states(row.as_strided((2, 1, 1, dim), (0, 0, 0, 1)),
                              torch.zeros(2, 1, 1, device="cuda"), out, lse_out=lo)
    assert torch.equal(out[0, 0], row)
    assert abs(float(lo) - 0.6931471805599453) < 2.0 ** -22
