"""Host-side checks of mla_prefill_attention, mla_latent_tree_attention and
mla_cache_compact_rows (no GPU needed, no kernel launched): every argument check refuses its
case with the documented status before any CUDA call, in the library and in the binding; empty
calls succeed; a valid call on a machine without a GPU fails with MLA_ERR_CUDA."""
import ctypes

import pytest
import torch

from pack_mla_cache_gb300 import build as B
from pack_mla_cache_gb300 import ops

A = 0x7F0000000000  # a 16-byte aligned fake device address (never dereferenced)
INV, UNS, MIS = ops.MLA_ERR_INVALID_ARG, ops.MLA_ERR_UNSUPPORTED, ops.MLA_ERR_MISALIGNED
BF16, I32 = torch.bfloat16, torch.int32
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the call without a GPU")


@pytest.fixture(scope="module")
def L():
    B.build()
    return ops.lib()


def refused(status, want, msg):
    assert status == want, ops.mla_last_error()
    assert msg in ops.mla_last_error()


# ------------------------------------------------------------------- prompts
def prefill(L, **kw):
    a = dict(qn=A, qnt=8 * 192, qnh=192, qp=A + 256, qpt=8 * 192, qph=192, dt=0, T=9, H=8, kn=A,
             knt=4 * 256, knh=256, kp=A, kpt=64, kph=0, v=A + 256, vt=4 * 256, vh=256, kd=0, K=20,
             G=4, N=128, P=64, V=128, cq=A, ck=A, S=2, scale=0.07, ks=None, causal=1, out=A,
             ot=8 * 128, oh=128, lse=A, lt=8, lh=1, ws=A, wsb=1 << 40, err=None)
    a.update(kw)
    return L.mla_prefill_attention(
        a["qn"], a["qnt"], a["qnh"], a["qp"], a["qpt"], a["qph"], a["dt"], a["T"], a["H"], a["kn"],
        a["knt"], a["knh"], a["kp"], a["kpt"], a["kph"], a["v"], a["vt"], a["vh"], a["kd"], a["K"],
        a["G"], a["N"], a["P"], a["V"], a["cq"], a["ck"], a["S"], a["scale"], a["ks"], a["causal"],
        a["out"], a["ot"], a["oh"], a["lse"], a["lt"], a["lh"], a["ws"], a["wsb"], a["err"], None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(T=-1), INV, "num_tokens"), (dict(K=-1), INV, "num_kv_tokens"), (dict(H=0), INV, "num_heads"),
    (dict(H=1028, G=4), UNS, "heads"), (dict(G=0), INV, "num_kv_heads"), (dict(G=3), INV, "num_kv_heads"),
    (dict(G=16), INV, "num_kv_heads"), (dict(S=0), INV, "num_seqs"), (dict(S=4097), UNS, "sequences"),
    (dict(T=1 << 29), UNS, "too large"), (dict(N=64), UNS, "nope_dim"), (dict(P=128), UNS, "rope_dim"),
    (dict(V=192), UNS, "v_dim"), (dict(dt=1), INV, "dtype must be"), (dict(dt=4), INV, "dtype must be"),
    (dict(kd=3), INV, "kv_dtype"), (dict(kd=4), INV, "kv_dtype"), (dict(dt=3), INV, "kv_dtype"),
    (dict(kd=1), INV, "require kv_scale"), (dict(ks=A), INV, "do not use kv_scale"),
    (dict(scale=float("inf")), INV, "softmax_scale"), (dict(scale=float("nan")), INV, "softmax_scale"),
    (dict(qn=A + 8), MIS, "q_nope"), (dict(qnt=8 * 192 + 4), MIS, "q_nope"), (dict(qnh=196), MIS, "q_nope"),
    (dict(qp=A + 2), MIS, "q_pe"), (dict(qpt=4), MIS, "q_pe"), (dict(kn=A + 8), MIS, "k_nope"),
    (dict(knh=260), MIS, "k_nope"), (dict(kpt=68), MIS, "k_pe"), (dict(kp=A + 4), MIS, "k_pe"),
    (dict(vt=1028), MIS, "v rows"), (dict(kd=1, ks=A, knt=8 * 257), MIS, "k_nope"),
    (dict(out=A + 4), MIS, "out rows"), (dict(oh=132), MIS, "out rows"),
    (dict(knt=0), UNS, "token strides"), (dict(vt=-1024), UNS, "token strides"),
    (dict(kpt=1 << 40), UNS, "token strides"), (dict(knh=-256), UNS, "head strides"),
    (dict(ws=A + 8), MIS, "workspace"), (dict(lse=A + 2), MIS, "4-byte"), (dict(cq=A + 1), MIS, "4-byte"),
    (dict(ck=A + 2), MIS, "4-byte"), (dict(err=A + 2), MIS, "4-byte"), (dict(kd=2, ks=A + 2), MIS, "4-byte"),
    (dict(qn=None), INV, "non-null"), (dict(qp=None), INV, "non-null"), (dict(cq=None), INV, "non-null"),
    (dict(ck=None), INV, "non-null"), (dict(out=None), INV, "non-null"), (dict(ws=None), INV, "non-null"),
    (dict(kn=None), INV, "non-null"), (dict(kp=None), INV, "non-null"), (dict(v=None), INV, "non-null"),
])
def test_prefill_refusals(L, kw, status, msg):
    refused(prefill(L, **kw), status, msg)


def test_prefill_empty(L):
    none = dict(qn=None, qp=None, kn=None, kp=None, v=None, cq=None, ck=None, out=None, ws=None, lse=None)
    assert prefill(L, T=0, **none) == ops.MLA_OK


@no_gpu
def test_without_a_gpu(L):
    assert prefill(L) == ops.MLA_ERR_CUDA
    assert tree(L) == ops.MLA_ERR_CUDA
    assert compact(L) == ops.MLA_ERR_CUDA
    n = ctypes.c_int64()
    assert L.mla_prefill_attention_workspace(9, 8, 4, 2, ctypes.byref(n)) == ops.MLA_ERR_CUDA


@pytest.mark.parametrize("args,status,msg", [
    ((-1, 8, 4, 2), INV, "num_tokens"), ((9, 0, 4, 2), INV, "num_heads"), ((9, 8, 3, 2), INV, "num_kv_heads"),
    ((9, 8, 4, 0), INV, "num_seqs"), ((1 << 30, 8, 4, 2), UNS, "too large"),
])
def test_prefill_workspace_refusals(L, args, status, msg):
    n = ctypes.c_int64()
    refused(L.mla_prefill_attention_workspace(*args, ctypes.byref(n)), status, msg)


def test_prefill_workspace_wants_a_place(L):
    refused(L.mla_prefill_attention_workspace(9, 8, 4, 2, None), INV, "bytes")


# ---------------------------------------------------------------------- trees
def tree(L, **kw):
    a = dict(T=8, H=16, kv=A, dtype=1, ks=A, mask=A, ms=2, mw=2, out=A, S=2)
    a.update(kw)
    return L.mla_latent_tree_attention(
        A, 16 * 576, 576, A + 1024, 16 * 576, 576, a["T"], a["H"], 512, 64, a["kv"], a["dtype"], 64, 64,
        64 * 576, 576, A, 32, A, A, a["S"], 0.07, a["ks"], a["mask"], a["ms"], a["mw"], a["out"], 16 * 512,
        512, A, 16, 1, A, 1 << 40, None, None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(mw=0), INV, "mask_words"), (dict(mw=1025), UNS, "drafted"), (dict(mask=A + 2), MIS, "tree_mask"),
    (dict(mask=None), INV, "tree_mask"), (dict(T=-1), INV, "num_tokens"), (dict(H=0), INV, "num_heads"),
    (dict(S=0), INV, "num_seqs"), (dict(dtype=3), INV, "cache_dtype"), (dict(ks=None), INV, "k_scale"),
    (dict(out=A + 8), MIS, "out rows"), (dict(kv=None), INV, "non-null"),
])
def test_tree_refusals(L, kw, status, msg):
    refused(tree(L, **kw), status, msg)


def test_tree_empty(L):
    assert tree(L, T=0, mask=None) == ops.MLA_OK


# ------------------------------------------------------------------ compaction
def compact(L, **kw):
    a = dict(ptrs=A, nl=5, dtype=1, nb=64, bs=64, bst=64 * 576, es=576, ed=576, bt=A, bts=8, st=A, rows=A,
             rs=9, mr=9, cnt=A, S=4, err=None)
    a.update(kw)
    return L.mla_cache_compact_rows(a["ptrs"], a["nl"], a["dtype"], a["nb"], a["bs"], a["bst"], a["es"],
                                    a["ed"], a["bt"], a["bts"], a["st"], a["rows"], a["rs"], a["mr"],
                                    a["cnt"], a["S"], a["err"], None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(S=-1), INV, "num_seqs"), (dict(nl=0), INV, "num_layers"), (dict(nl=129), UNS, "128 layers"),
    (dict(dtype=3), INV, "cache_dtype"), (dict(bs=0), INV, "block_size"), (dict(nb=0), INV, "num_blocks"),
    (dict(bts=0), INV, "block_table_stride"), (dict(ed=0), INV, "entry_dim"), (dict(ed=592), INV, "entry_dim"),
    (dict(bst=63 * 576), INV, "block_stride"), (dict(mr=-1), INV, "max_rows"), (dict(mr=1025), UNS, "1024 rows"),
    (dict(es=584, bst=64 * 584), MIS, "entry_stride"), (dict(bst=64 * 576 + 8), MIS, "block_stride"),
    (dict(ed=568), MIS, "entry_dim"), (dict(ptrs=A + 4), MIS, "kv_cache_ptrs"), (dict(bt=A + 2), MIS, "index arrays"),
    (dict(st=A + 1), MIS, "index arrays"), (dict(rows=A + 2), MIS, "index arrays"), (dict(cnt=A + 3), MIS, "index arrays"),
    (dict(err=A + 2), MIS, "err_word"), (dict(S=1 << 31 >> 1, nl=128), UNS, "too large"),
    (dict(ptrs=None), INV, "non-null"), (dict(bt=None), INV, "non-null"), (dict(st=None), INV, "non-null"),
    (dict(rows=None), INV, "non-null"), (dict(cnt=None), INV, "non-null"),
])
def test_compact_refusals(L, kw, status, msg):
    refused(compact(L, **kw), status, msg)


def test_compact_empty(L):
    none = dict(ptrs=None, bt=None, st=None, rows=None, cnt=None)
    assert compact(L, S=0, **none) == ops.MLA_OK
    assert compact(L, mr=0, **none) == ops.MLA_OK


# --------------------------------------------------------------------- binding
def call_prefill(**kw):
    T, H, K, G, S = 6, 4, 10, 2, 3
    q, both = torch.zeros(T, H, 192, dtype=BF16), torch.zeros(K, G, 256, dtype=BF16)
    a = dict(q_nope=q[:, :, :128], q_pe=q[:, :, 128:], k_nope=both[:, :, :128],
             k_pe=torch.zeros(K, 64, dtype=BF16), v=both[:, :, 128:], cu_q_lens=torch.zeros(S + 1, dtype=I32),
             cu_kv_lens=torch.zeros(S + 1, dtype=I32), out=torch.zeros(T, H, 128, dtype=BF16),
             workspace=torch.zeros(64, dtype=torch.uint8), softmax_scale=1.0, lse=torch.zeros(T, H), stream=0)
    a.update(kw)
    ops.mla_prefill_attention(**a)


@pytest.mark.parametrize("kw,msg", [
    (dict(q_pe=torch.zeros(6, 4, 64)), "dtype"), (dict(out=torch.zeros(6, 4, 128)), "dtype"),
    (dict(k_pe=torch.zeros(10, 64)), "dtype"), (dict(v=torch.zeros(10, 2, 128)), "dtype"),
    (dict(q_pe=torch.zeros(5, 4, 64, dtype=BF16)), "q_pe must be"), (dict(k_pe=torch.zeros(9, 64, dtype=BF16)), "k_pe must be"),
    (dict(k_pe=torch.zeros(10, 1, 64, dtype=BF16)), "k_pe must be"), (dict(v=torch.zeros(10, 1, 128, dtype=BF16)), "v must be"),
    (dict(k_nope=torch.zeros(10, 2, 64, dtype=BF16)), "k_nope must be"),
    (dict(out=torch.zeros(6, 4, 64, dtype=BF16)), "out must be"), (dict(lse=torch.zeros(4, 6)), "lse must be"),
    (dict(v=torch.zeros(10, 2, 256, dtype=BF16)[:, :, ::2]), "unit last stride"),
    (dict(q_nope=torch.zeros(6, 4, 256, dtype=BF16)[:, :, ::2]), "unit last stride"),
    (dict(cu_q_lens=torch.zeros(4, dtype=torch.int64)), "cu_q_lens must be"),
    (dict(cu_kv_lens=torch.zeros(3, dtype=I32)), "cu_kv_lens must be"),
    (dict(kv_scale=torch.ones(1, dtype=torch.float64)), "kv_scale must be"),
    (dict(workspace=torch.zeros(64, 2, dtype=torch.uint8)[:, 0]), "workspace must be"),
])
def test_prefill_binding_refuses(kw, msg):
    with pytest.raises(ValueError, match=msg):
        call_prefill(**kw)


@pytest.mark.parametrize("kw", [
    dict(), dict(lse=None), dict(k_pe=torch.zeros(10, 2, 64, dtype=BF16)),
    dict(k_nope=torch.zeros(10, 1, 128, dtype=BF16).expand(10, 2, 128)), dict(lse=torch.zeros(4, 6).t()),
])
def test_prefill_binding_forwards(kw):
    """Host tensors of the right form pass the binding and are refused by the library."""
    with pytest.raises(ops.MlaError):
        call_prefill(**kw)


def call_tree(**kw):
    T, H, S = 4, 2, 3
    q = torch.zeros(T, H, 576, dtype=BF16)
    a = dict(q_c=q[:, :, :512], q_pe=q[:, :, 512:], kv_cache=torch.zeros(8 * 16 * 576, dtype=torch.uint8),
             cache_dtype=1, num_blocks=8, block_size=16, block_stride=16 * 576, entry_stride=576,
             block_table=torch.zeros(S, 5, dtype=I32), cu_q_lens=torch.zeros(S + 1, dtype=I32),
             kv_lens=torch.zeros(S, dtype=I32), tree_mask=torch.zeros(T, 2, dtype=I32),
             out=torch.zeros(T, H, 512, dtype=BF16), workspace=torch.zeros(64, dtype=torch.uint8),
             softmax_scale=1.0, k_scale=torch.ones(1), lse=torch.zeros(T, H), stream=0)
    a.update(kw)
    ops.mla_latent_tree_attention(**a)


@pytest.mark.parametrize("kw,msg", [
    (dict(tree_mask=torch.zeros(4, 2, dtype=torch.int64)), "tree_mask must be"),
    (dict(tree_mask=torch.zeros(3, 2, dtype=I32)), "tree_mask must be"),
    (dict(tree_mask=torch.zeros(8, dtype=I32)), "tree_mask must be"),
    (dict(tree_mask=torch.zeros(2, 4, dtype=I32).t()), "tree_mask must be"),
    (dict(q_pe=torch.zeros(4, 1, 64, dtype=BF16)), "q_pe must be"), (dict(out=torch.zeros(3, 2, 512, dtype=BF16)), "out must be"),
    (dict(kv_lens=torch.zeros(3, dtype=torch.int64)), "kv_lens must be"),
])
def test_tree_binding_refuses(kw, msg):
    with pytest.raises(ValueError, match=msg):
        call_tree(**kw)


@pytest.mark.parametrize("kw", [dict(), dict(tree_mask=torch.zeros(4, 9, dtype=I32)[:, :2]),
                                dict(tree_mask=torch.zeros(1, 4, dtype=I32).t())])
def test_tree_binding_forwards(kw):
    with pytest.raises(ops.MlaError):
        call_tree(**kw)


def call_compact(**kw):
    a = dict(kv_cache_ptrs=torch.zeros(2, dtype=torch.int64), cache_dtype=1, num_blocks=8, block_size=16,
             block_stride=16 * 576, entry_stride=576, entry_dim=576, block_table=torch.zeros(3, 5, dtype=I32),
             starts=torch.zeros(3, dtype=I32), rows=torch.zeros(3, 4, dtype=I32), counts=torch.zeros(3, dtype=I32), stream=0)
    a.update(kw)
    ops.mla_cache_compact_rows(**a)


@pytest.mark.parametrize("kw,msg", [
    (dict(kv_cache_ptrs=torch.zeros(2, dtype=I32)), "kv_cache_ptrs must be"), (dict(starts=torch.zeros(3)), "starts must be"),
    (dict(counts=torch.zeros(2, dtype=I32)), "counts must be"), (dict(rows=torch.zeros(2, 4, dtype=I32)), "rows must be"),
    (dict(rows=torch.zeros(4, 3, dtype=I32).t()), "rows must be"), (dict(block_table=torch.zeros(3, 5)), "block_table must be"),
])
def test_compact_binding_refuses(kw, msg):
    with pytest.raises(ValueError, match=msg):
        call_compact(**kw)


def test_compact_binding_forwards():
    with pytest.raises(ops.MlaError):
        call_compact()
