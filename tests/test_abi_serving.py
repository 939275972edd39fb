"""Host-side checks of the serving operators (no GPU needed, no kernel
launched): every argument check of mla_cache_copy_blocks, mla_latent_attention
and mla_merge_attn_states rejects its case with the documented status before
any CUDA call; empty calls succeed; a valid call on a machine without a GPU
fails with MLA_ERR_CUDA."""
import ctypes

import pytest
import torch

from pack_mla_cache_gb300 import build as B
from pack_mla_cache_gb300 import ops

A = 0x7F0000000000  # a 16-byte aligned fake device address (never dereferenced)
INV, UNS, MIS = ops.MLA_ERR_INVALID_ARG, ops.MLA_ERR_UNSUPPORTED, ops.MLA_ERR_MISALIGNED
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the call without a GPU")


@pytest.fixture(scope="module")
def L():
    B.build()
    return ops.lib()


def refused(L, status, want, msg):
    assert status == want, ops.mla_last_error()
    assert msg in ops.mla_last_error()


# ------------------------------------------------------------------ block copies
def copy(L, **kw):
    a = dict(ptrs=A, nl=5, dtype=1, nb=64, bs=64, bst=64 * 576, es=576, ed=576, src=A + 64,
             dst=A + 128, rows=A + 192, n=4, err=None)
    a.update(kw)
    return L.mla_cache_copy_blocks(a["ptrs"], a["nl"], a["dtype"], a["nb"], a["bs"], a["bst"],
                                   a["es"], a["ed"], a["src"], a["dst"], a["rows"], a["n"],
                                   a["err"], None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(n=-1), INV, "num_copies"), (dict(nl=0), INV, "num_layers"),
    (dict(nl=129), UNS, "128 layers"), (dict(dtype=3), INV, "cache_dtype"),
    (dict(dtype=4), INV, "cache_dtype"), (dict(bs=0), INV, "block_size"),
    (dict(nb=0), INV, "num_blocks"), (dict(ed=0), INV, "entry_dim"),
    (dict(ed=592), INV, "entry_dim"), (dict(bst=63 * 576), INV, "block_stride"),
    (dict(bst=-(1 << 62), es=1 << 61), INV, "block_stride"),
    (dict(es=584, bst=64 * 584), MIS, "entry_stride"), (dict(bst=64 * 576 + 8), MIS, "block_stride"),
    (dict(ed=568), MIS, "entry_dim"), (dict(bs=1 << 27, bst=(1 << 27) * 576), UNS, "32 GiB"),
    (dict(ptrs=A + 4), MIS, "kv_cache_ptrs"), (dict(src=A + 2), MIS, "index arrays"),
    (dict(rows=A + 1), MIS, "index arrays"), (dict(err=A + 2), MIS, "err_word"),
    (dict(ptrs=None), INV, "non-null"), (dict(src=None), INV, "non-null"),
    (dict(dst=None), INV, "non-null"),
])
def test_copy_blocks_refusals(L, kw, status, msg):
    refused(L, copy(L, **kw), status, msg)


def test_copy_blocks_empty(L):
    assert copy(L, n=0, ptrs=None, src=None, dst=None, rows=None) == ops.MLA_OK


# ------------------------------------------------------------------- attention
def attend(L, **kw):
    a = dict(qc=A, qct=16 * 576, qch=576, qp=A + 1024, qpt=16 * 576, qph=576, T=8, H=16, R=512,
             P=64, kv=A, dtype=1, nb=64, bs=64, bst=64 * 576, es=576, bt=A, bts=32, cu=A, kvl=A,
             S=2, scale=0.07, ks=A, causal=1, out=A, ot=16 * 512, oh=512, lse=A, lt=16, lh=1,
             ws=A, wsb=1 << 40, err=None)
    a.update(kw)
    return L.mla_latent_attention(
        a["qc"], a["qct"], a["qch"], a["qp"], a["qpt"], a["qph"], a["T"], a["H"], a["R"], a["P"],
        a["kv"], a["dtype"], a["nb"], a["bs"], a["bst"], a["es"], a["bt"], a["bts"], a["cu"],
        a["kvl"], a["S"], a["scale"], a["ks"], a["causal"], a["out"], a["ot"], a["oh"], a["lse"],
        a["lt"], a["lh"], a["ws"], a["wsb"], a["err"], None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(T=-1), INV, "num_tokens"), (dict(H=0), INV, "num_heads"), (dict(H=1025), UNS, "heads"),
    (dict(S=0), INV, "num_seqs"), (dict(S=4097), UNS, "sequences"),
    (dict(T=1 << 30, H=16), UNS, "too large"), (dict(R=256), UNS, "kv_lora_rank"),
    (dict(P=32), UNS, "pe_dim"), (dict(dtype=3), INV, "cache_dtype"),
    (dict(dtype=4), INV, "cache_dtype"), (dict(ks=None), INV, "requires k_scale"),
    (dict(dtype=0), INV, "does not use k_scale"), (dict(scale=float("nan")), INV, "softmax_scale"),
    (dict(scale=float("inf")), INV, "softmax_scale"), (dict(bs=0), INV, "block_size"),
    (dict(nb=0), INV, "num_blocks"), (dict(bts=0), INV, "block_table_stride"),
    (dict(es=560), INV, "entry_stride"), (dict(bst=63 * 576), INV, "block_stride"),
    (dict(es=584, bst=64 * 584), MIS, "cache rows"), (dict(kv=A + 8), MIS, "cache rows"),
    (dict(bt=A + 2), MIS, "index arrays"), (dict(kvl=A + 1), MIS, "index arrays"),
    (dict(qc=A + 2), MIS, "q_c"), (dict(qct=577), MIS, "q_c"), (dict(qph=68), MIS, "q_pe"),
    (dict(out=A + 8), MIS, "out"), (dict(oh=516), MIS, "out"), (dict(ws=A + 4), MIS, "workspace"),
    (dict(lse=A + 2), MIS, "lse"), (dict(ks=A + 1), MIS, "k_scale"), (dict(err=A + 2), MIS, "err_word"),
    (dict(qc=None), INV, "non-null"), (dict(qp=None), INV, "non-null"),
    (dict(kv=None), INV, "non-null"), (dict(bt=None), INV, "non-null"),
    (dict(cu=None), INV, "non-null"), (dict(kvl=None), INV, "non-null"),
    (dict(out=None), INV, "non-null"), (dict(ws=None), INV, "non-null"),
])
def test_latent_attention_refusals(L, kw, status, msg):
    refused(L, attend(L, **kw), status, msg)


def test_latent_attention_empty(L):
    assert attend(L, T=0, qc=None, qp=None, out=None, ws=None, lse=None) == ops.MLA_OK


def test_latent_attention_workspace_refusals(L):
    n = ctypes.c_int64(0)
    f = L.mla_latent_attention_workspace
    refused(L, f(-1, 16, 1, ctypes.byref(n)), INV, "num_tokens")
    refused(L, f(1, 0, 1, ctypes.byref(n)), INV, "num_heads")
    refused(L, f(1, 1025, 1, ctypes.byref(n)), UNS, "heads")
    refused(L, f(1, 16, 0, ctypes.byref(n)), INV, "num_seqs")
    refused(L, f(1, 16, 5000, ctypes.byref(n)), UNS, "sequences")
    refused(L, f(1, 16, 1, None), INV, "bytes")


# ----------------------------------------------------------------------- merge
def merge(L, **kw):
    a = dict(parts=A, ps=1 << 20, ts=16 * 512, hs=512, lse=A, lps=128, lts=16, lhs=1, dtype=0,
             P=2, T=8, H=16, D=512, out=A, ot=16 * 512, oh=512, lo=A, lot=16, loh=1)
    a.update(kw)
    return L.mla_merge_attn_states(
        a["parts"], a["ps"], a["ts"], a["hs"], a["lse"], a["lps"], a["lts"], a["lhs"], a["dtype"],
        a["P"], a["T"], a["H"], a["D"], a["out"], a["ot"], a["oh"], a["lo"], a["lot"], a["loh"],
        None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(T=-1), INV, "num_tokens"), (dict(H=0), INV, "num_heads"), (dict(P=0), INV, "num_parts"),
    (dict(P=1025), UNS, "parts"), (dict(D=0), INV, "dim"), (dict(dtype=1), INV, "dtype"),
    (dict(dtype=2), INV, "dtype"), (dict(dtype=5), INV, "dtype"), (dict(D=12), MIS, "dim"),
    (dict(dtype=4, D=6), MIS, "dim"), (dict(parts=A + 8), MIS, "parts"), (dict(ps=4), MIS, "parts"),
    (dict(ts=100), MIS, "parts"), (dict(oh=4), MIS, "out"), (dict(out=A + 2), MIS, "out"),
    (dict(lse=A + 2), MIS, "lse"), (dict(lo=A + 1), MIS, "lse_out"),
    (dict(parts=None), INV, "non-null"), (dict(lse=None), INV, "non-null"),
    (dict(out=None), INV, "non-null"),
])
def test_merge_refusals(L, kw, status, msg):
    refused(L, merge(L, **kw), status, msg)


def test_merge_empty(L):
    assert merge(L, T=0, parts=None, lse=None, out=None) == ops.MLA_OK


def test_merge_binding_refuses_mixed_types(L):
    p = torch.zeros(2, 1, 1, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dtype"):
        ops.mla_merge_attn_states(p, torch.zeros(2, 1, 1), torch.zeros(1, 1, 8))


# -------------------------------------------------------------------- no device
@no_gpu
def test_without_a_gpu(L):
    assert copy(L) == ops.MLA_ERR_CUDA
    assert attend(L) == ops.MLA_ERR_CUDA
    assert merge(L) == ops.MLA_ERR_CUDA
    n = ctypes.c_int64(0)
    assert L.mla_latent_attention_workspace(1, 16, 1, ctypes.byref(n)) == ops.MLA_ERR_CUDA


def test_attention_timeout_hook(L):
    assert L.mla_test_attention_timeout(1000, 2) == 0
    assert L.mla_test_attention_timeout(0, 0) == 0  # defaults back
