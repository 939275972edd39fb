"""The Python binding of the serving operators refuses tensors that the C interface would
read as something else (no GPU needed: nothing is launched)."""
import pytest
import torch

from pack_mla_cache_gb300 import ops

BF16, I32 = torch.bfloat16, torch.int32


def attend(**kw):
    T, H, S = 4, 2, 3
    q = torch.zeros(T, H, 576, dtype=BF16)
    a = dict(q_c=q[:, :, :512], q_pe=q[:, :, 512:], kv_cache=torch.zeros(8 * 16 * 576, dtype=torch.uint8),
             cache_dtype=1, num_blocks=8, block_size=16, block_stride=16 * 576, entry_stride=576,
             block_table=torch.zeros(S, 5, dtype=I32), cu_q_lens=torch.zeros(S + 1, dtype=I32),
             kv_lens=torch.zeros(S, dtype=I32), out=torch.zeros(T, H, 512, dtype=BF16),
             workspace=torch.zeros(64, dtype=torch.uint8), softmax_scale=1.0,
             k_scale=torch.ones(1), lse=torch.zeros(T, H), stream=0)
    a.update(kw)
    ops.mla_latent_attention(**a)


@pytest.mark.parametrize("kw,msg", [
    (dict(q_c=torch.zeros(4, 2, 512, dtype=torch.float16)), "must be bf16"),
    (dict(q_pe=torch.zeros(4, 2, 64)), "must be bf16"),
    (dict(out=torch.zeros(4, 2, 512, dtype=torch.float16)), "must be bf16"),
    (dict(q_c=torch.zeros(4, 2, 1024, dtype=BF16)[:, :, ::2]), "unit last stride"),
    (dict(q_pe=torch.zeros(4, 64, 2, dtype=BF16).transpose(1, 2)), "unit last stride"),
    (dict(out=torch.zeros(4, 512, 2, dtype=BF16).transpose(1, 2)), "unit last stride"),
    (dict(q_pe=torch.zeros(3, 2, 64, dtype=BF16)), "q_pe must be"),
    (dict(q_pe=torch.zeros(4, 1, 64, dtype=BF16)), "q_pe must be"),
    (dict(out=torch.zeros(3, 2, 512, dtype=BF16)), "out must be"),
    (dict(out=torch.zeros(4, 2, 64, dtype=BF16)), "out must be"),
    (dict(lse=torch.zeros(4, 2, dtype=torch.float64)), "lse must be"),
    (dict(lse=torch.zeros(2, 4)), "lse must be"),
    (dict(kv_lens=torch.zeros(3, dtype=torch.int64)), "kv_lens must be"),
    (dict(kv_lens=torch.zeros(6, dtype=I32)[::2]), "kv_lens must be"),
    (dict(cu_q_lens=torch.zeros(4, dtype=torch.int64)), "cu_q_lens must be"),
    (dict(cu_q_lens=torch.zeros(3, dtype=I32)), "cu_q_lens must be"),
    (dict(block_table=torch.zeros(3, 5, dtype=torch.int64)), "block_table must be"),
    (dict(block_table=torch.zeros(2, 5, dtype=I32)), "block_table must be"),
    (dict(block_table=torch.zeros(15, dtype=I32)), "block_table must be"),
    (dict(block_table=torch.zeros(5, 3, dtype=I32).t()), "block_table must be"),
    (dict(k_scale=torch.ones(1, dtype=torch.float64)), "k_scale must be"),
    (dict(k_scale=torch.ones(0)), "k_scale must be"),
    (dict(workspace=torch.zeros(64, 2, dtype=torch.uint8)[:, 0]), "workspace must be"),
])
def test_attention_refuses(kw, msg):
    with pytest.raises(ValueError, match=msg):
        attend(**kw)


@pytest.mark.parametrize("kw", [
    dict(), dict(lse=None), dict(block_table=torch.zeros(4, 5, dtype=I32)),
    dict(lse=torch.zeros(2, 4).t()), dict(q_c=torch.zeros(1, 1, 512, dtype=BF16).expand(4, 2, 512)),
    dict(block_table=torch.zeros(3, 9, dtype=I32)[:, :5]), dict(cu_q_lens=torch.zeros(9, dtype=I32)),
    dict(block_table=torch.zeros(1, 3, dtype=I32).t()), dict(k_scale=torch.ones(1).expand(4)),
    dict(k_scale=torch.tensor(1.0)),
])
def test_attention_forwards_what_the_interface_takes(kw):
    """Host tensors of the right form pass the binding and are refused by the library."""
    with pytest.raises(ops.MlaError):
        attend(**kw)


def merge(**kw):
    a = dict(parts=torch.zeros(2, 3, 4, 8), lse=torch.zeros(2, 3, 4), out=torch.zeros(3, 4, 8),
             lse_out=torch.zeros(3, 4), stream=0)
    a.update(kw)
    ops.mla_merge_attn_states(**a)


@pytest.mark.parametrize("kw,msg", [
    (dict(out=torch.zeros(3, 4, 8, dtype=BF16)), "dtype"),
    (dict(out=torch.zeros(3, 4, 16)), "out must be"), (dict(out=torch.zeros(2, 4, 8)), "out must be"),
    (dict(parts=torch.zeros(2, 3, 8, 4).transpose(2, 3)), "unit last stride"),
    (dict(out=torch.zeros(3, 8, 4).transpose(1, 2)), "unit last stride"),
    (dict(lse=torch.zeros(2, 3, 4, dtype=BF16)), "lse must be"), (dict(lse=torch.zeros(2, 4, 3)), "lse must be"),
    (dict(lse_out=torch.zeros(3, 4, dtype=torch.float64)), "lse_out must be"),
    (dict(lse_out=torch.zeros(4, 3)), "lse_out must be"),
])
def test_merge_refuses(kw, msg):
    with pytest.raises(ValueError, match=msg):
        merge(**kw)


def test_merge_forwards_what_the_interface_takes():
    for kw in (dict(), dict(lse_out=None), dict(lse=torch.zeros(2, 4, 3).transpose(1, 2))):
        with pytest.raises(ops.MlaError):
            merge(**kw)


def copy(**kw):
    i = lambda n: torch.zeros(n, dtype=I32)
    a = dict(kv_cache_ptrs=torch.zeros(2, dtype=torch.int64), cache_dtype=1, num_blocks=8,
             block_size=16, block_stride=16 * 576, entry_stride=576, entry_dim=576, src_blocks=i(3),
             dst_blocks=i(3), row_counts=i(3), stream=0)
    a.update(kw)
    ops.mla_cache_copy_blocks(**a)


@pytest.mark.parametrize("kw,msg", [
    (dict(kv_cache_ptrs=torch.zeros(2, dtype=I32)), "kv_cache_ptrs must be"),
    (dict(kv_cache_ptrs=torch.zeros(4, dtype=torch.int64)[::2]), "kv_cache_ptrs must be"),
    (dict(src_blocks=torch.zeros(3, dtype=torch.int64)), "src_blocks must be"),
    (dict(src_blocks=torch.zeros(2, dtype=I32)), "src_blocks must be"),
    (dict(dst_blocks=torch.zeros(3, dtype=torch.int64)), "dst_blocks must be"),
    (dict(dst_blocks=torch.zeros(6, dtype=I32)[::2]), "dst_blocks must be"),
    (dict(row_counts=torch.zeros(2, dtype=I32)), "row_counts must be"),
    (dict(row_counts=torch.zeros(3, dtype=torch.int64)), "row_counts must be"),
])
def test_copy_refuses(kw, msg):
    with pytest.raises(ValueError, match=msg):
        copy(**kw)


def test_copy_forwards_what_the_interface_takes():
    for kw in (dict(), dict(row_counts=None)):
        with pytest.raises(ops.MlaError):
            copy(**kw)


def test_the_current_stream_without_the_private_call(monkeypatch):
    """On a torch without the raw handle's call the public stream object is asked."""
    class Stream:
        cuda_stream = 1234
    monkeypatch.setattr(ops, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream())
    assert ops._stream(None) == 1234
    assert ops._stream(Stream()) == 1234 and ops._stream(7) == 7


@pytest.mark.gpu
def test_the_current_stream_is_the_one_torch_names():
    s = torch.cuda.Stream()
    assert ops._stream(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(s):
        assert ops._stream(None) == s.cuda_stream == torch.cuda.current_stream().cuda_stream


def test_lists_count_their_elements(monkeypatch):
    """A list as a row [1, n] is n elements (its first extent alone dropped the others)."""
    seen = {}

    class Lib:
        @staticmethod
        def mla_cache_copy_blocks(*a):
            seen["copy"] = (a[1], a[11])
            return 0

        @staticmethod
        def mla_latent_attention(*a):
            seen["seqs"] = a[20]
            return 0
    monkeypatch.setattr(ops, "lib", lambda: Lib)
    copy(kv_cache_ptrs=torch.zeros(1, 2, dtype=torch.int64), dst_blocks=torch.zeros(1, 3, dtype=I32))
    attend(kv_lens=torch.zeros(1, 3, dtype=I32))
    assert seen == {"copy": (2, 3), "seqs": 3}
