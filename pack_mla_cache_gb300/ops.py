"""Thin Python binding of libmla_cache (include/mla_cache.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Each function has the name of the C entry point it calls, takes
torch tensors (device memory) and forwards their data pointers, element
strides and the current CUDA stream.  A failing call raises ``MlaError`` with
the library's status and message.  There is no fallback: if the library is
not built, ``lib()`` raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

from .build import LIB_PATH

MLA_BF16, MLA_FP8_E4M3, MLA_FP8_E5M2, MLA_FP16, MLA_FP32 = 0, 1, 2, 3, 4
MLA_OK, MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED, MLA_ERR_MISALIGNED, MLA_ERR_CUDA = range(5)
MLA_ERRBIT_SLOT_OOB, MLA_ERRBIT_BLOCK_OOB, MLA_ERRBIT_POS_OOB, MLA_ERRBIT_MISALIGNED = 1, 2, 4, 8
MLA_ERRBIT_TIMEOUT = 16

_TORCH_DTYPE = {MLA_BF16: torch.bfloat16, MLA_FP8_E4M3: torch.float8_e4m3fn,
                MLA_FP8_E5M2: torch.float8_e5m2, MLA_FP16: torch.float16}


class MlaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[mla status {status}] {message}")
        self.status = status


class KvPack(ctypes.Structure):
    _fields_ = [("k_nope", ctypes.c_void_p), ("kn_token_stride", ctypes.c_int64),
                ("kn_head_stride", ctypes.c_int64), ("v", ctypes.c_void_p),
                ("v_token_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("in_dtype", ctypes.c_int), ("k_pe", ctypes.c_void_p),
                ("kpe_token_stride", ctypes.c_int64), ("kpe_dtype", ctypes.c_int),
                ("num_tokens", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("nope_dim", ctypes.c_int32), ("rope_dim", ctypes.c_int32),
                ("v_dim", ctypes.c_int32), ("key_out", ctypes.c_void_p),
                ("v_out", ctypes.c_void_p), ("out_dtype", ctypes.c_int),
                ("out_scale", ctypes.c_void_p)]


class ContextGather(ctypes.Structure):
    _fields_ = [("kv_cache", ctypes.c_void_p), ("cache_dtype", ctypes.c_int),
                ("num_blocks", ctypes.c_int64), ("block_size", ctypes.c_int32),
                ("block_stride", ctypes.c_int64), ("entry_stride", ctypes.c_int64),
                ("entry_dim", ctypes.c_int32), ("block_table", ctypes.c_void_p),
                ("block_table_stride", ctypes.c_int64), ("cu_chunk_lens", ctypes.c_void_p),
                ("chunk_starts", ctypes.c_void_p), ("num_seqs", ctypes.c_int32),
                ("num_tokens", ctypes.c_int32), ("out", ctypes.c_void_p),
                ("out_row_stride", ctypes.c_int64), ("out_dtype", ctypes.c_int)]


class NormRope(ctypes.Structure):
    _fields_ = [("gamma", ctypes.c_void_p), ("gamma_layer_stride", ctypes.c_int64),
                ("eps", ctypes.c_float), ("positions", ctypes.c_void_p),
                ("cos_sin_cache", ctypes.c_void_p), ("max_position", ctypes.c_int64)]


_lib = None

# C signatures of every entry point declared in include/mla_cache.h
_i32, _i64, _u32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p
SIGNATURES = {
    "mla_dtype_from_string": (ctypes.c_int, [ctypes.c_char_p]),
    "mla_last_error": (ctypes.c_char_p, []),
    "mla_version": (ctypes.c_char_p, []),
    "mla_set_pdl": (ctypes.c_int, [ctypes.c_int]),
    "mla_set_bulk_copy": (ctypes.c_int, [ctypes.c_int]),
    "mla_set_pointer_checks": (ctypes.c_int, [ctypes.c_int]),
    "mla_set_gather_early_tables": (ctypes.c_int, [ctypes.c_int]),
    "mla_set_insert_early_tables": (ctypes.c_int, [ctypes.c_int]),
    "mla_test_insert_timeout": (ctypes.c_int, [ctypes.c_uint64, _i64]),
    "mla_test_attention_timeout": (ctypes.c_int, [ctypes.c_uint64, _i32]),
    "mla_cache_insert_grouped": (ctypes.c_int, [
        _vp, _i64, _i64, _vp, _i64, _i64, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _vp,
        ctypes.c_int, _i64, _i32, _i64, _i64, ctypes.POINTER(NormRope), _vp, _vp]),
    "mla_context_gather": (ctypes.c_int, [
        _vp, ctypes.c_int, _i64, _i32, _i64, _i64, _i32, _vp, _i64, _vp, _vp, _i32, _i32, _vp,
        _i64, ctypes.c_int, _vp, _vp]),
    "mla_context_kv_pack": (ctypes.c_int, [
        _vp, _i64, _i64, _vp, _i64, _i64, ctypes.c_int, _vp, _i64, ctypes.c_int, _i32, _i32, _i32,
        _i32, _i32, _vp, _vp, ctypes.c_int, _vp, _vp, _vp]),
    "mla_context_gather_scaled": (ctypes.c_int, [
        _vp, ctypes.c_int, _i64, _i32, _i64, _i64, _i32, _vp, _i64, _vp, _vp, _i32, _i32, _vp,
        _i64, _vp, _vp, _vp]),
    "mla_context_kv_pack_paged": (ctypes.c_int, [
        _vp, _i64, _i64, _vp, _i64, _i64, ctypes.c_int, _vp, ctypes.c_int, _i64, _i32, _i64, _i64,
        _i64, _vp,
        _i64, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp, ctypes.c_int, _vp, _vp,
        _vp]),
    "mla_norm_rope_grouped": (ctypes.c_int, [
        _vp, _i64, _i64, _vp, _i64, _i64, _i32, _i32, _i32, _i32, ctypes.POINTER(NormRope), _vp,
        _i64, _i64, _vp, _i64, _i64, _vp, _vp]),
    "mla_rope_cos_sin_cache": (ctypes.c_int, [_vp, _i64, _i32, ctypes.c_double, _vp]),
    "mla_context_kv_pack_gather": (ctypes.c_int, [ctypes.POINTER(KvPack),
                                                  ctypes.POINTER(ContextGather), _vp, _vp]),
    "mla_cache_copy_blocks": (ctypes.c_int, [
        _vp, _i32, ctypes.c_int, _i64, _i32, _i64, _i64, _i32, _vp, _vp, _vp, _i32, _vp, _vp]),
    "mla_latent_attention": (ctypes.c_int, [
        _vp, _i64, _i64, _vp, _i64, _i64, _i32, _i32, _i32, _i32, _vp, ctypes.c_int, _i64, _i32,
        _i64, _i64, _vp, _i64, _vp, _vp, _i32, ctypes.c_float, _vp, _i32, _vp, _i64, _i64, _vp,
        _i64, _i64, _vp, _i64, _vp, _vp]),
    "mla_latent_tree_attention": (ctypes.c_int, [
        _vp, _i64, _i64, _vp, _i64, _i64, _i32, _i32, _i32, _i32, _vp, ctypes.c_int, _i64, _i32,
        _i64, _i64, _vp, _i64, _vp, _vp, _i32, ctypes.c_float, _vp, _vp, _i64, _i32, _vp, _i64,
        _i64, _vp, _i64, _i64, _vp, _i64, _vp, _vp]),
    "mla_cache_compact_rows": (ctypes.c_int, [
        _vp, _i32, ctypes.c_int, _i64, _i32, _i64, _i64, _i32, _vp, _i64, _vp, _vp, _i64, _i32, _vp,
        _i32, _vp, _vp]),
    "mla_prefill_attention": (ctypes.c_int, [
        _vp, _i64, _i64, _vp, _i64, _i64, ctypes.c_int, _i32, _i32, _vp, _i64, _i64, _vp, _i64, _i64,
        _vp, _i64, _i64, ctypes.c_int, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _i32, ctypes.c_float,
        _vp, _i32, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _vp]),
    "mla_prefill_attention_workspace": (ctypes.c_int, [_i32, _i32, _i32, _i32,
                                                       ctypes.POINTER(_i64)]),
    "mla_latent_attention_workspace": (ctypes.c_int, [_i32, _i32, _i32, ctypes.POINTER(_i64)]),
    "mla_merge_attn_states": (ctypes.c_int, [
        _vp, _i64, _i64, _i64, _vp, _i64, _i64, _i64, ctypes.c_int, _i32, _i32, _i32, _i32, _vp,
        _i64, _i64, _vp, _i64, _i64, _vp]),
}


def lib() -> ctypes.CDLL:
    """Load libmla_cache.so (built in-tree by pack_mla_cache_gb300.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libmla_cache.so is not built ({LIB_PATH} missing): run "
                "pack_mla_cache_gb300.build.build() first; there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int) -> None:
    if status != MLA_OK:
        raise MlaError(status, lib().mla_last_error().decode())


_CODES = {v: k for k, v in _TORCH_DTYPE.items()}


def dtype_code(d) -> int:
    code = _CODES.get(d)  # most calls name a torch dtype
    if code is not None:
        return code
    if isinstance(d, int):
        return d
    if isinstance(d, torch.dtype):
        for k, v in _TORCH_DTYPE.items():
            if v == d:
                return k
        raise ValueError(f"unsupported dtype {d}")
    code = lib().mla_dtype_from_string(str(d).encode())
    if code < 0:
        raise MlaError(MLA_ERR_INVALID_ARG, f"unknown kv cache dtype string {d!r}")
    return code


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


# The current stream's handle alone (a Stream object costs 3 us).  Not part of torch's
# public interface: a torch without it goes the public way.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def mla_dtype_from_string(s: str) -> int:
    return lib().mla_dtype_from_string(s.encode())


def mla_last_error() -> str:
    return lib().mla_last_error().decode()


def mla_version() -> str:
    return lib().mla_version().decode()


def mla_set_pdl(enable: bool) -> bool:
    return bool(lib().mla_set_pdl(1 if enable else 0))


def mla_set_bulk_copy(mode: int) -> int:
    """0 never, 1 large calls (default), 2 every call whose layout qualifies;
    returns the previous mode."""
    return int(lib().mla_set_bulk_copy(int(mode)))


def mla_set_pointer_checks(enable: bool) -> bool:
    """Switch the per-call device-pointer checks on (default) or off; returns
    the previous setting."""
    return bool(lib().mla_set_pointer_checks(1 if enable else 0))


def mla_set_gather_early_tables(enable: bool) -> bool:
    """Let the context gathers read their tables before the programmatic
    launch wait (the tables must be complete before each call is enqueued);
    returns the previous setting."""
    return bool(lib().mla_set_gather_early_tables(1 if enable else 0))


def mla_set_insert_early_tables(enable: bool) -> bool:
    """Let the grouped insert read kv_cache_ptrs and kv_scales before the
    programmatic launch wait (both must be complete before each call is
    enqueued); returns the previous setting."""
    return bool(lib().mla_set_insert_early_tables(1 if enable else 0))


def mla_test_insert_timeout(wait_limit_ns: int = 0, skip_item: int = -1) -> None:
    """Testing hook of the insert's bulk-copy pipeline (see the C header);
    ``mla_test_insert_timeout()`` restores the defaults."""
    lib().mla_test_insert_timeout(int(wait_limit_ns), int(skip_item))


def mla_test_attention_timeout(wait_limit_ns: int = 0, stall_stage: int = 0) -> None:
    """Testing hook for the attention's bounded waits (see mla_cache.h);
    ``mla_test_attention_timeout()`` restores the defaults."""
    lib().mla_test_attention_timeout(int(wait_limit_ns), int(stall_stage))


def mla_cache_insert_grouped(kv_c, k_pe, slot_mapping, kv_cache_ptrs, kv_scales, cache_dtype,
                             num_blocks, block_size, block_stride, entry_stride, *,
                             slot_layer_stride=None, gamma=None, eps=1e-6, positions=None,
                             cos_sin_cache=None, err_word=None, stream=None):
    """kv_c [L, T, R] and k_pe [L, T, P] bf16 views (any strides, unit last
    stride); slot_mapping int64 [L, T] or [T] (shared); kv_cache_ptrs int64 [L];
    kv_scales fp32 [L] or None."""
    L, T, R = kv_c.shape
    P = k_pe.shape[2]
    if slot_layer_stride is None:
        slot_layer_stride = 0 if slot_mapping.dim() == 1 else slot_mapping.stride(0)
    nr = None
    if gamma is not None or positions is not None:
        nr = NormRope(_ptr(gamma), 0 if gamma is None else gamma.stride(0), float(eps),
                      _ptr(positions), _ptr(cos_sin_cache),
                      0 if cos_sin_cache is None else cos_sin_cache.shape[0])
    _check(lib().mla_cache_insert_grouped(
        _ptr(kv_c), kv_c.stride(1), kv_c.stride(0), _ptr(k_pe), k_pe.stride(1), k_pe.stride(0),
        T, L, R, P, _ptr(slot_mapping), slot_layer_stride, _ptr(kv_cache_ptrs), _ptr(kv_scales),
        dtype_code(cache_dtype), num_blocks, block_size, block_stride, entry_stride,
        ctypes.byref(nr) if nr is not None else None, _ptr(err_word), _stream(stream)))


def mla_norm_rope_grouped(kv_c, k_pe, kv_c_out, k_pe_out, *, gamma=None, eps=1e-6,
                          positions=None, cos_sin_cache=None, err_word=None, stream=None):
    """Every tensor is a bf16 view indexed [token, layer, i] (any strides, unit
    last stride): kv_c / kv_c_out [T, L, 512], k_pe / k_pe_out [T, L, 64].  For
    layer-major outputs pass e.g. ``out.transpose(0, 1)`` of an [L, T, .] tensor."""
    T, L, R = kv_c.shape
    P = k_pe.shape[2]
    nr = None
    if gamma is not None or positions is not None:
        nr = NormRope(_ptr(gamma), 0 if gamma is None else gamma.stride(0), float(eps),
                      _ptr(positions), _ptr(cos_sin_cache),
                      0 if cos_sin_cache is None else cos_sin_cache.shape[0])
    _check(lib().mla_norm_rope_grouped(
        _ptr(kv_c), kv_c.stride(0), kv_c.stride(1), _ptr(k_pe), k_pe.stride(0), k_pe.stride(1),
        T, L, R, P, ctypes.byref(nr) if nr is not None else None, _ptr(kv_c_out),
        kv_c_out.stride(0), kv_c_out.stride(1), _ptr(k_pe_out), k_pe_out.stride(0),
        k_pe_out.stride(1), _ptr(err_word), _stream(stream)))


def mla_context_gather(kv_cache, cache_dtype, num_blocks, block_size, block_stride,
                       entry_stride, entry_dim, block_table, cu_chunk_lens, chunk_starts, out,
                       out_dtype, *, num_tokens=None, err_word=None, stream=None):
    """kv_cache: the cache base (any tensor over its bytes); block_table int32
    [S, W]; out [num_tokens, >= entry_dim] with unit last stride."""
    S = chunk_starts.shape[0]
    n = out.shape[0] if num_tokens is None else num_tokens
    _check(lib().mla_context_gather(
        _ptr(kv_cache), dtype_code(cache_dtype), num_blocks, block_size, block_stride,
        entry_stride, entry_dim, _ptr(block_table), _bt_stride(block_table), _ptr(cu_chunk_lens),
        _ptr(chunk_starts), S, n, _ptr(out), out.stride(0), dtype_code(out_dtype),
        _ptr(err_word), _stream(stream)))


def _bt_stride(block_table):
    # row width of the table: its row stride (a one-row table's stride is not
    # meaningful, so its width is used)
    return block_table.stride(0) if block_table.size(0) > 1 else block_table.size(1)


def mla_context_gather_scaled(kv_cache, cache_dtype, num_blocks, block_size, block_stride,
                              entry_stride, entry_dim, block_table, cu_chunk_lens, chunk_starts,
                              out, k_scale, *, num_tokens=None, err_word=None, stream=None):
    """The gather with the fp8 -> bf16 widening times ``k_scale`` (device fp32
    scalar tensor); out is bf16 [num_tokens, >= entry_dim]."""
    S = chunk_starts.shape[0]
    n = out.shape[0] if num_tokens is None else num_tokens
    _check(lib().mla_context_gather_scaled(
        _ptr(kv_cache), dtype_code(cache_dtype), num_blocks, block_size, block_stride,
        entry_stride, entry_dim, _ptr(block_table), _bt_stride(block_table),
        _ptr(cu_chunk_lens), _ptr(chunk_starts), S, n, _ptr(out), out.stride(0), _ptr(k_scale),
        _ptr(err_word), _stream(stream)))


def mla_context_kv_pack_paged(k_nope, v, kv_cache, cache_dtype, num_blocks, block_size,
                              block_stride, entry_stride, block_table, cu_chunk_lens,
                              chunk_starts, key_out, v_out, out_dtype, *, rope_offset=512,
                              rope_dim=64, out_scale=None, in_dtype=None, err_word=None,
                              stream=None):
    """The pack with each token's k_pe read from its paged cache row at
    ``rope_offset``; k_nope / v [T, H, 128] bf16 views (strided)."""
    T, H, N = k_nope.shape
    _check(lib().mla_context_kv_pack_paged(
        _ptr(k_nope), k_nope.stride(0), k_nope.stride(1), _ptr(v), v.stride(0), v.stride(1),
        dtype_code(in_dtype if in_dtype is not None else k_nope.dtype), _ptr(kv_cache),
        dtype_code(cache_dtype), num_blocks, block_size, block_stride,
        entry_stride, rope_offset, _ptr(block_table), _bt_stride(block_table),
        _ptr(cu_chunk_lens), _ptr(chunk_starts), chunk_starts.shape[0], T, H, N, rope_dim,
        v.shape[2], _ptr(key_out), _ptr(v_out), dtype_code(out_dtype), _ptr(out_scale),
        _ptr(err_word), _stream(stream)))


def mla_context_kv_pack(k_nope, v, k_pe, key_out, v_out, out_dtype, *, kpe_dtype=None,
                        out_scale=None, in_dtype=None, err_word=None, stream=None):
    """k_nope / v: [T, H, 128] bf16 or fp16 views (strided; their dtype is the
    input type unless ``in_dtype`` is given); k_pe [T, 64] (the input type or
    fp8, strided rows); key_out [T, H, 192] and v_out [T, H, 128] (or None)."""
    T, H, N = k_nope.shape
    kd = dtype_code(kpe_dtype if kpe_dtype is not None else k_pe.dtype)
    _check(lib().mla_context_kv_pack(
        _ptr(k_nope), k_nope.stride(0), k_nope.stride(1), _ptr(v), v.stride(0), v.stride(1),
        dtype_code(in_dtype if in_dtype is not None else k_nope.dtype), _ptr(k_pe),
        k_pe.stride(0), kd, T, H, N, k_pe.shape[-1], v.shape[2], _ptr(key_out),
        _ptr(v_out), dtype_code(out_dtype), _ptr(out_scale), _ptr(err_word), _stream(stream)))


def mla_rope_cos_sin_cache(out, base=10000.0, *, stream=None):
    """Fill out (fp32 [max_position, rot_dim]) with the rotary cos/sin table."""
    _check(lib().mla_rope_cos_sin_cache(_ptr(out), out.shape[0], out.shape[1], float(base),
                                        _stream(stream)))


def kv_pack_desc(k_nope, v, k_pe, key_out, v_out, out_dtype, *, kpe_dtype=None, out_scale=None,
                 in_dtype=None) -> KvPack:
    """The arguments of ``mla_context_kv_pack`` as the C struct."""
    T, H, N = k_nope.shape
    return KvPack(_ptr(k_nope), k_nope.stride(0), k_nope.stride(1), _ptr(v), v.stride(0),
                  v.stride(1), dtype_code(in_dtype if in_dtype is not None else k_nope.dtype),
                  _ptr(k_pe), k_pe.stride(0),
                  dtype_code(kpe_dtype if kpe_dtype is not None else k_pe.dtype), T, H, N,
                  k_pe.shape[-1], v.shape[2], _ptr(key_out), _ptr(v_out), dtype_code(out_dtype),
                  _ptr(out_scale))


def context_gather_desc(kv_cache, cache_dtype, num_blocks, block_size, block_stride,
                        entry_stride, entry_dim, block_table, cu_chunk_lens, chunk_starts, out,
                        out_dtype, *, num_tokens=None) -> ContextGather:
    """The arguments of ``mla_context_gather`` as the C struct."""
    n = out.shape[0] if num_tokens is None else num_tokens
    return ContextGather(_ptr(kv_cache), dtype_code(cache_dtype), num_blocks, block_size,
                         block_stride, entry_stride, entry_dim, _ptr(block_table),
                         _bt_stride(block_table), _ptr(cu_chunk_lens), _ptr(chunk_starts),
                         chunk_starts.shape[0], n, _ptr(out), out.stride(0),
                         dtype_code(out_dtype))


def mla_context_kv_pack_gather(pack: KvPack, next_gather: ContextGather, *, err_word=None,
                               stream=None):
    """One launch: the pack described by ``pack`` (``kv_pack_desc``) and the
    gather described by ``next_gather`` (``context_gather_desc``); the gather
    must write a workspace the pack does not use."""
    _check(lib().mla_context_kv_pack_gather(ctypes.byref(pack), ctypes.byref(next_gather),
                                            _ptr(err_word), _stream(stream)))


# (The checks' usual path is a few attribute reads: a small call's time is its host work.)
def _is_list(t, dtype, n):
    # at least n elements of the type, one behind the other
    return t.dtype is dtype and t.numel() >= n and t.is_contiguous()


def _refuse(name, t, want):
    raise ValueError(f"{name} must be {want} (got {t.dtype} {list(t.shape)}, strides {t.stride()})")


def mla_cache_copy_blocks(kv_cache_ptrs, cache_dtype, num_blocks, block_size, block_stride,
                          entry_stride, entry_dim, src_blocks, dst_blocks, *, row_counts=None,
                          err_word=None, stream=None):
    """Copy (fork, compact) or clear (src -1) blocks in every layer's cache:
    kv_cache_ptrs int64 [L]; src_blocks / dst_blocks / row_counts int32 [N],
    row_counts None for whole blocks."""
    N, L = dst_blocks.numel(), kv_cache_ptrs.numel()
    if not _is_list(kv_cache_ptrs, torch.int64, L):
        _refuse("kv_cache_ptrs", kv_cache_ptrs, "contiguous int64")
    if not _is_list(dst_blocks, torch.int32, N):
        _refuse("dst_blocks", dst_blocks, "contiguous int32")
    if not _is_list(src_blocks, torch.int32, N):
        _refuse("src_blocks", src_blocks, f"contiguous int32 [{N}]")
    if row_counts is not None and not _is_list(row_counts, torch.int32, N):
        _refuse("row_counts", row_counts, f"contiguous int32 [{N}]")
    _check(lib().mla_cache_copy_blocks(
        _ptr(kv_cache_ptrs), L, dtype_code(cache_dtype), num_blocks,
        block_size, block_stride, entry_stride, entry_dim, _ptr(src_blocks), _ptr(dst_blocks),
        _ptr(row_counts), N, _ptr(err_word), _stream(stream)))


def mla_latent_attention_workspace(num_tokens: int, num_heads: int, num_seqs: int) -> int:
    """Bytes of workspace of ``mla_latent_attention`` on the current device."""
    n = _i64(0)
    _check(lib().mla_latent_attention_workspace(num_tokens, num_heads, num_seqs, ctypes.byref(n)))
    return n.value


def _latent_args(q_c, q_pe, kv_lens, cu_q_lens, block_table, k_scale, out, lse, workspace):
    """Checks what both attentions over the latent cache take; strides and sizes of it."""
    T, H, R = q_c.shape
    qc_t, qc_h, qc_e = q_c.stride()
    qp_t, qp_h, qp_e = q_pe.stride()
    out_t, out_h, out_e = out.stride()
    S = kv_lens.numel()
    bf16 = torch.bfloat16
    qp_T, qp_H, P = q_pe.shape
    if q_c.dtype is not bf16 or q_pe.dtype is not bf16 or out.dtype is not bf16:
        raise ValueError(f"q_c, q_pe and out must be bf16 (got {q_c.dtype}, {q_pe.dtype}, {out.dtype})")
    if qc_e != 1 or qp_e != 1 or out_e != 1:
        raise ValueError("q_c, q_pe and out must have a unit last stride")
    if qp_T != T or qp_H != H:
        _refuse("q_pe", q_pe, f"[{T}, {H}, 64]")
    if out.shape != (T, H, R):
        _refuse("out", out, f"[{T}, {H}, {R}]")
    lse_t = lse_h = 0
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (T, H):
            _refuse("lse", lse, f"fp32 [{T}, {H}]")
        lse_t, lse_h = lse.stride()
    if not _is_list(kv_lens, torch.int32, S):
        _refuse("kv_lens", kv_lens, "contiguous int32")
    if not _is_list(cu_q_lens, torch.int32, S + 1):
        _refuse("cu_q_lens", cu_q_lens, f"contiguous int32 [{S + 1}]")
    if block_table.dtype is not torch.int32 or block_table.ndim != 2:
        _refuse("block_table", block_table, f"int32 [{S}, W]")
    tab_S, tab_W = block_table.shape
    tab_s, tab_e = block_table.stride()
    if (tab_e != 1 and tab_W > 1) or tab_S < S:
        _refuse("block_table", block_table, f"int32 [{S}, W] with a unit last stride")
    if k_scale is not None and (k_scale.dtype is not torch.float32 or k_scale.numel() < 1):
        _refuse("k_scale", k_scale, "an fp32 scalar")
    if not workspace.is_contiguous():
        _refuse("workspace", workspace, "contiguous")
    return (T, H, R, P, S, qc_t, qc_h, qp_t, qp_h, out_t, out_h, lse_t, lse_h,
            tab_s if tab_S > 1 else tab_W)


def mla_latent_attention(q_c, q_pe, kv_cache, cache_dtype, num_blocks, block_size, block_stride,
                         entry_stride, block_table, cu_q_lens, kv_lens, out, workspace, *,
                         softmax_scale, k_scale=None, causal=True, lse=None, err_word=None,
                         stream=None):
    """Attention of new tokens over the paged latent cache (absorbed form):
    q_c [T, H, 512] and q_pe [T, H, 64] bf16 views (any strides, unit last
    stride), out bf16 [T, H, 512] likewise, lse fp32 [T, H] or None; block_table
    int32 [S, W] (a slice of a wider table is as wide as its row stride),
    cu_q_lens int32 [S + 1], kv_lens int32 [S]; k_scale fp32;
    workspace: a uint8 tensor of ``mla_latent_attention_workspace`` bytes."""
    T, H, R, P, S, qc_t, qc_h, qp_t, qp_h, out_t, out_h, lse_t, lse_h, width = _latent_args(
        q_c, q_pe, kv_lens, cu_q_lens, block_table, k_scale, out, lse, workspace)
    status = lib().mla_latent_attention(
        q_c.data_ptr(), qc_t, qc_h, q_pe.data_ptr(), qp_t, qp_h, T, H, R, P,
        kv_cache.data_ptr(), dtype_code(cache_dtype), num_blocks, block_size, block_stride,
        entry_stride, block_table.data_ptr(), width, cu_q_lens.data_ptr(),
        kv_lens.data_ptr(), S, softmax_scale, _ptr(k_scale), 1 if causal else 0,
        out.data_ptr(), out_t, out_h, _ptr(lse), lse_t, lse_h, workspace.data_ptr(),
        workspace.nbytes, _ptr(err_word), _stream(stream))
    if status:
        _check(status)


def mla_latent_tree_attention(q_c, q_pe, kv_cache, cache_dtype, num_blocks, block_size,
                              block_stride, entry_stride, block_table, cu_q_lens, kv_lens,
                              tree_mask, out, workspace, *, softmax_scale, k_scale=None, lse=None,
                              err_word=None, stream=None):
    """``mla_latent_attention`` for trees of drafted tokens: tree_mask int32 [T, W] (any row
    stride, unit last stride); bit i % 32 of word i // 32 says that the token sees the row of
    its sequence's new token i.  The context before the new tokens is seen by all."""
    T, H, R, P, S, qc_t, qc_h, qp_t, qp_h, out_t, out_h, lse_t, lse_h, width = _latent_args(
        q_c, q_pe, kv_lens, cu_q_lens, block_table, k_scale, out, lse, workspace)
    if tree_mask.dtype is not torch.int32 or tree_mask.ndim != 2 or tree_mask.shape[0] != T or \
            (tree_mask.shape[1] > 1 and tree_mask.stride(1) != 1):
        _refuse("tree_mask", tree_mask, f"int32 [{T}, W] with a unit last stride")
    status = lib().mla_latent_tree_attention(
        q_c.data_ptr(), qc_t, qc_h, q_pe.data_ptr(), qp_t, qp_h, T, H, R, P,
        kv_cache.data_ptr(), dtype_code(cache_dtype), num_blocks, block_size, block_stride,
        entry_stride, block_table.data_ptr(), width, cu_q_lens.data_ptr(),
        kv_lens.data_ptr(), S, softmax_scale, _ptr(k_scale), tree_mask.data_ptr(),
        tree_mask.stride(0), tree_mask.shape[1], out.data_ptr(), out_t, out_h, _ptr(lse), lse_t,
        lse_h, workspace.data_ptr(), workspace.nbytes, _ptr(err_word), _stream(stream))
    if status:
        _check(status)


def mla_cache_compact_rows(kv_cache_ptrs, cache_dtype, num_blocks, block_size, block_stride,
                           entry_stride, entry_dim, block_table, starts, rows, counts, *,
                           err_word=None, stream=None):
    """Move accepted rows to the front of the drafted ones in every layer's cache: row
    ``starts[s] + i`` becomes row ``starts[s] + rows[s, i]`` for i < counts[s]; kv_cache_ptrs
    int64 [L], block_table int32 [S, W], starts / counts int32 [S], rows int32 [S, N] (each
    list strictly increasing)."""
    L, S = kv_cache_ptrs.numel(), starts.numel()
    if not _is_list(kv_cache_ptrs, torch.int64, L):
        _refuse("kv_cache_ptrs", kv_cache_ptrs, "contiguous int64")
    if not _is_list(starts, torch.int32, S):
        _refuse("starts", starts, "contiguous int32")
    if not _is_list(counts, torch.int32, S):
        _refuse("counts", counts, f"contiguous int32 [{S}]")
    if block_table.dtype is not torch.int32 or block_table.ndim != 2:
        _refuse("block_table", block_table, f"int32 [{S}, W]")
    tab_S, tab_W = block_table.shape
    tab_s, tab_e = block_table.stride()
    if (tab_e != 1 and tab_W > 1) or tab_S < S:
        _refuse("block_table", block_table, f"int32 [{S}, W] with a unit last stride")
    if rows.dtype is not torch.int32 or rows.ndim != 2:
        _refuse("rows", rows, f"int32 [{S}, N]")
    rows_S, width = rows.shape
    rows_s, rows_e = rows.stride()
    if (rows_e != 1 and width > 1) or rows_S < S:
        _refuse("rows", rows, f"int32 [{S}, N] with a unit last stride")
    status = lib().mla_cache_compact_rows(
        kv_cache_ptrs.data_ptr(), L, dtype_code(cache_dtype), num_blocks, block_size, block_stride,
        entry_stride, entry_dim, block_table.data_ptr(), tab_s if tab_S > 1 else tab_W,
        starts.data_ptr(), rows.data_ptr(), rows_s, width, counts.data_ptr(), S, _ptr(err_word),
        _stream(stream))
    if status:
        _check(status)


def mla_prefill_attention_workspace(num_tokens: int, num_heads: int, num_kv_heads: int,
                                    num_seqs: int) -> int:
    """Bytes of workspace of ``mla_prefill_attention`` on the current device."""
    n = _i64(0)
    _check(lib().mla_prefill_attention_workspace(num_tokens, num_heads, num_kv_heads, num_seqs,
                                                 ctypes.byref(n)))
    return n.value


def mla_prefill_attention(q_nope, q_pe, k_nope, k_pe, v, cu_q_lens, cu_kv_lens, out, workspace, *,
                          softmax_scale, causal=True, kv_scale=None, lse=None, err_word=None,
                          stream=None):
    """Attention of packed sequences over keys and values per head: q_nope [T, H, 128] and
    q_pe [T, H, 64] (bf16 or fp16), k_nope [K, G, 128], k_pe [K, G, 64] or [K, 64] (shared by
    all heads) and v [K, G, 128] (q's type, or fp8 with ``kv_scale`` an fp32 scalar), out
    [T, H, 128] of q's type, lse fp32 [T, H] or None; any strides with a unit last one;
    cu_q_lens and cu_kv_lens int32 [S + 1]; workspace: a uint8 tensor of
    ``mla_prefill_attention_workspace`` bytes."""
    T, H, N = q_nope.shape
    K, G, kn_N = k_nope.shape
    qp_T, qp_H, P = q_pe.shape
    v_K, v_G, V = v.shape
    qn_t, qn_h, qn_e = q_nope.stride()
    qp_t, qp_h, qp_e = q_pe.stride()
    kn_t, kn_h, kn_e = k_nope.stride()
    v_t, v_h, v_e = v.stride()
    out_t, out_h, out_e = out.stride()
    if k_pe.ndim == 2:
        (kp_K, kp_P), (kp_t, kp_e) = k_pe.shape, k_pe.stride()
        kp_G, kp_h = G, 0
    else:
        (kp_K, kp_G, kp_P), (kp_t, kp_h, kp_e) = k_pe.shape, k_pe.stride()
    qd, kd = q_nope.dtype, k_nope.dtype
    if q_pe.dtype is not qd or out.dtype is not qd:
        raise ValueError(f"q_pe and out must have q_nope's dtype ({qd}, got {q_pe.dtype}, {out.dtype})")
    if k_pe.dtype is not kd or v.dtype is not kd:
        raise ValueError(f"k_pe and v must have k_nope's dtype ({kd}, got {k_pe.dtype}, {v.dtype})")
    if qp_T != T or qp_H != H:
        _refuse("q_pe", q_pe, f"[{T}, {H}, 64]")
    if kp_K != K or kp_G != G or kp_P != P:
        _refuse("k_pe", k_pe, f"[{K}, {P}] or [{K}, {G}, {P}]")
    if kn_N != N:
        _refuse("k_nope", k_nope, f"[{K}, {G}, {N}]")
    if v_K != K or v_G != G:
        _refuse("v", v, f"[{K}, {G}, 128]")
    if out.shape != (T, H, V):
        _refuse("out", out, f"[{T}, {H}, {V}]")
    if not qn_e == qp_e == kn_e == kp_e == v_e == out_e == 1:
        raise ValueError("q_nope, q_pe, k_nope, k_pe, v and out must have a unit last stride")
    lse_t = lse_h = 0
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (T, H):
            _refuse("lse", lse, f"fp32 [{T}, {H}]")
        lse_t, lse_h = lse.stride()
    S = cu_q_lens.numel() - 1
    if not _is_list(cu_q_lens, torch.int32, 2):
        _refuse("cu_q_lens", cu_q_lens, "contiguous int32 [S + 1]")
    if not _is_list(cu_kv_lens, torch.int32, S + 1):
        _refuse("cu_kv_lens", cu_kv_lens, f"contiguous int32 [{S + 1}]")
    if kv_scale is not None and (kv_scale.dtype is not torch.float32 or kv_scale.numel() < 1):
        _refuse("kv_scale", kv_scale, "an fp32 scalar")
    if not workspace.is_contiguous():
        _refuse("workspace", workspace, "contiguous")
    status = lib().mla_prefill_attention(
        q_nope.data_ptr(), qn_t, qn_h, q_pe.data_ptr(), qp_t, qp_h, dtype_code(qd), T, H,
        k_nope.data_ptr(), kn_t, kn_h, k_pe.data_ptr(), kp_t, kp_h, v.data_ptr(), v_t, v_h,
        dtype_code(kd), K, G, N, P, V, cu_q_lens.data_ptr(), cu_kv_lens.data_ptr(), S,
        softmax_scale, _ptr(kv_scale), 1 if causal else 0, out.data_ptr(), out_t, out_h, _ptr(lse),
        lse_t, lse_h, workspace.data_ptr(), workspace.nbytes, _ptr(err_word), _stream(stream))
    if status:
        _check(status)


def mla_merge_attn_states(parts, lse, out, *, lse_out=None, stream=None):
    """Join attention results over disjoint parts of the context: parts
    [P, T, H, D] (bf16, fp16 or fp32; any strides, unit last stride) with lse fp32
    [P, T, H] into out [T, H, D] of the same type and lse_out fp32 [T, H]."""
    P, T, H, Dm = parts.shape
    p_p, p_t, p_h, p_e = parts.stride()
    out_t, out_h, out_e = out.stride()
    lo_t = lo_h = 0
    if parts.dtype != out.dtype:
        raise ValueError(f"out must have the parts' dtype ({parts.dtype}, got {out.dtype})")
    if out.shape != (T, H, Dm):
        _refuse("out", out, f"[{T}, {H}, {Dm}]")
    if p_e != 1 or out_e != 1:
        raise ValueError("parts and out must have a unit last stride")
    if lse.dtype is not torch.float32 or lse.shape != (P, T, H):
        _refuse("lse", lse, f"fp32 [{P}, {T}, {H}]")
    if lse_out is not None:
        if lse_out.dtype is not torch.float32 or lse_out.shape != (T, H):
            _refuse("lse_out", lse_out, f"fp32 [{T}, {H}]")
        lo_t, lo_h = lse_out.stride()
    lse_p, lse_t, lse_h = lse.stride()
    code = MLA_FP32 if parts.dtype == torch.float32 else dtype_code(parts.dtype)
    _check(lib().mla_merge_attn_states(
        parts.data_ptr(), p_p, p_t, p_h, lse.data_ptr(), lse_p, lse_t, lse_h, code, P, T, H, Dm,
        out.data_ptr(), out_t, out_h, _ptr(lse_out), lo_t, lo_h, _stream(stream)))
