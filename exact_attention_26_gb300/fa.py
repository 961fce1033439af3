"""Thin ctypes binding over libfa.so, with the C ABI's names.

Argument marshalling only: every step of the attention computation runs in the
library's CUDA kernels.  torch supplies device memory and the current stream.
There is no CPU path; a missing library or a non-CUDA tensor raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import math
import os

import torch

from . import build as _build

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_MISALIGNED = 3
FA_ERR_CUDA = 4
FA_ERR_TIMEOUT = 5
FA_ERR_WORKSPACE = 6
FA_ERR_BAD_INDEX = 7

EXPORTED = ("fa_fwd", "fa_bwd", "fa_bwd_workspace_bytes", "fa_status_string", "fa_device_status",
            "fa_selftest_wait_timeout", "fa_decode", "fa_decode_num_splits",
            "fa_decode_uses_tensor_cores",
            "fa_decode_workspace_bytes", "fa_decode_paged", "fa_decode_paged_num_splits",
            "fa_decode_paged_workspace_bytes", "fa_fwd_gqa", "fa_bwd_gqa", "fa_fwd_varlen",
            "fa_bwd_varlen", "fa_quantize_fp8_workspace_bytes", "fa_quantize_fp8", "fa_fwd_fp8",
            "fa_probe_unit_rates", "fa_probe_read_bandwidth", "fa_fwd_ws", "fa_fwd_workspace_bytes",
            "fa_fwd_split_segments", "fa_append_paged_fp8", "fa_decode_paged_fp8",
            "fa_decode_paged_fp8_workspace_bytes", "fa_free_pages", "fa_fork_pages",
            "fa_compact_pages", "fa_copy_pages", "fa_decode_paged_tree",
            "fa_decode_paged_tree_workspace_bytes", "fa_verify_tree", "fa_keep_path")

_vp = ctypes.c_void_p
_int = ctypes.c_int
_LIB = None
_NATIVE = None


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fa_status_string(status)} (status {status})")


def lib_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load libfa.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it first (__graft_entry__.build())")
        lib = ctypes.CDLL(path)
        lib.fa_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _int, _int, _int, _int, _int,
                               ctypes.c_float, _vp]
        lib.fa_fwd.restype = _int
        lib.fa_bwd_workspace_bytes.argtypes = [_int, _int, _int, _int]
        lib.fa_bwd_workspace_bytes.restype = ctypes.c_size_t
        lib.fa_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _int, _int,
                               _int, _int, ctypes.c_float, _vp, ctypes.c_size_t, _vp]
        lib.fa_bwd.restype = _int
        lib.fa_status_string.argtypes = [_int]
        lib.fa_status_string.restype = ctypes.c_char_p
        lib.fa_device_status.argtypes = [_vp]
        lib.fa_device_status.restype = _int
        lib.fa_fwd_gqa.argtypes = [_vp] * 5 + [_int] * 6 + [ctypes.c_float, _vp]
        lib.fa_fwd_gqa.restype = _int
        lib.fa_bwd_gqa.argtypes = [_vp] * 9 + [_int] * 6 + [ctypes.c_float, _vp, ctypes.c_size_t, _vp]
        lib.fa_bwd_gqa.restype = _int
        lib.fa_fwd_varlen.argtypes = [_vp] * 6 + [_int] * 7 + [ctypes.c_float, _vp]
        lib.fa_fwd_varlen.restype = _int
        lib.fa_bwd_varlen.argtypes = [_vp] * 10 + [_int] * 7 + [ctypes.c_float, _vp, ctypes.c_size_t,
                                                                 _vp]
        lib.fa_bwd_varlen.restype = _int
        lib.fa_quantize_fp8_workspace_bytes.argtypes = [_int] * 3
        lib.fa_quantize_fp8_workspace_bytes.restype = ctypes.c_size_t
        lib.fa_quantize_fp8.argtypes = [_vp] * 3 + [_int] * 4 + [_vp, _int, _vp, ctypes.c_size_t, _vp]
        lib.fa_quantize_fp8.restype = _int
        lib.fa_fwd_fp8.argtypes = [_vp] * 8 + [_int] * 6 + [ctypes.c_float, _vp]
        lib.fa_fwd_fp8.restype = _int
        lib.fa_decode.argtypes = [_vp] * 5 + [_int] * 6 + [ctypes.c_float, _int, _vp,
                                                          ctypes.c_size_t, _vp]
        lib.fa_decode.restype = _int
        lib.fa_decode_num_splits.argtypes = [_int] * 7
        lib.fa_decode_num_splits.restype = _int
        lib.fa_decode_uses_tensor_cores.argtypes = [_int] * 5
        lib.fa_decode_uses_tensor_cores.restype = _int
        lib.fa_decode_workspace_bytes.argtypes = [_int] * 7
        lib.fa_decode_workspace_bytes.restype = ctypes.c_size_t
        lib.fa_decode_paged.argtypes = [_vp] * 7 + [_int] * 8 + [ctypes.c_float, _int, _vp,
                                                                ctypes.c_size_t, _vp]
        lib.fa_decode_paged.restype = _int
        lib.fa_decode_paged_num_splits.argtypes = [_int] * 8
        lib.fa_decode_paged_num_splits.restype = _int
        lib.fa_decode_paged_workspace_bytes.argtypes = [_int] * 8
        lib.fa_decode_paged_workspace_bytes.restype = ctypes.c_size_t
        lib.fa_append_paged_fp8.argtypes = [_vp] * 9 + [_int] * 8 + [ctypes.c_longlong] * 2 + [_vp]
        lib.fa_append_paged_fp8.restype = _int
        lib.fa_decode_paged_fp8_workspace_bytes.argtypes = [_int] * 7
        lib.fa_decode_paged_fp8_workspace_bytes.restype = ctypes.c_size_t
        lib.fa_decode_paged_fp8.argtypes = [_vp] * 9 + [_int] * 10 + [ctypes.c_float, _vp,
                                                                    ctypes.c_size_t, _vp]
        lib.fa_decode_paged_fp8.restype = _int
        lib.fa_free_pages.argtypes = [_vp] * 4 + [_int] * 4 + [_vp]
        lib.fa_free_pages.restype = _int
        lib.fa_fork_pages.argtypes = [_vp] * 8 + [_int] * 5 + [_vp]
        lib.fa_fork_pages.restype = _int
        lib.fa_compact_pages.argtypes = [_vp] * 6 + [_int] * 4 + [_vp]
        lib.fa_compact_pages.restype = _int
        lib.fa_copy_pages.argtypes = [_vp, _vp, _int, _int, _vp, _vp, _int, _vp, _vp]
        lib.fa_copy_pages.restype = _int
        lib.fa_decode_paged_tree_workspace_bytes.argtypes = [_int] * 8
        lib.fa_decode_paged_tree_workspace_bytes.restype = ctypes.c_size_t
        lib.fa_decode_paged_tree.argtypes = [_vp] * 8 + [_int] * 9 + [ctypes.c_float, _vp,
                                                                     ctypes.c_size_t, _vp]
        lib.fa_decode_paged_tree.restype = _int
        lib.fa_verify_tree.argtypes = [_vp] * 8 + [_int] * 5 + [_vp]
        lib.fa_verify_tree.restype = _int
        lib.fa_keep_path.argtypes = [_vp, _int] + [_vp] * 5 + [_int] * 7 + [_vp]
        lib.fa_keep_path.restype = _int
        _LIB = lib
    return _LIB


def native():
    """The CPython extension that makes the paged-cache calls on tensors (raises if it has
    not been built)."""
    global _NATIVE
    if _NATIVE is None:
        load()
        if not os.path.exists(_build.EXT):
            raise RuntimeError(f"{_build.EXT} is missing: build it first (__graft_entry__.build())")
        loader = importlib.machinery.ExtensionFileLoader("_fa_torch", _build.EXT)
        spec = importlib.util.spec_from_file_location("_fa_torch", _build.EXT, loader=loader)
        _NATIVE = importlib.util.module_from_spec(spec)
    return _NATIVE


# ------------------------------------------------------------ raw C-ABI calls

def fa_fwd(q, k, v, o, lse, B, H, N, d, causal, scale, stream) -> int:
    return load().fa_fwd(q, k, v, o, lse, B, H, N, d, int(bool(causal)), scale, stream)


def fa_bwd_workspace_bytes(B, H, N, d) -> int:
    return load().fa_bwd_workspace_bytes(B, H, N, d)


def fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, H, N, d, causal, scale, workspace,
           workspace_bytes, stream) -> int:
    return load().fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, H, N, d, int(bool(causal)),
                         scale, workspace, workspace_bytes, stream)


def fa_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, B, H, N, d, causal, scale,
                   stream) -> int:
    """fa_bwd without a workspace: the library's fixed scratch array is used instead."""
    fn = load().fa_bwd_noalloc
    if fn.argtypes is None:
        fn.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _int, _int, _int, _int,
                       ctypes.c_float, _vp]
        fn.restype = _int
    return fn(q, k, v, o, lse, dout, dq, dk, dv, B, H, N, d, int(bool(causal)), scale, stream)


def fa_selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    """Run the bounded-wait self test (a wait nothing satisfies, limited to limit_ns)."""
    fn = load().fa_selftest_wait_timeout
    if fn.argtypes is None:
        fn.argtypes = [ctypes.c_ulonglong, _vp]
        fn.restype = _int
    return fn(limit_ns, stream)


def fa_probe_unit_rates(rates, iters: int, stream=None) -> int:
    """Run the unit-rate probes; `rates` is a ctypes array of 3 doubles (host)."""
    fn = load().fa_probe_unit_rates
    if fn.argtypes is None:
        fn.argtypes = [ctypes.POINTER(ctypes.c_double), _int, _vp]
        fn.restype = _int
    return fn(rates, iters, stream)


def fa_probe_read_bandwidth(buf, nbytes: int, iters: int, stream, gbs) -> int:
    """Time streaming reads of nbytes at device pointer buf; `gbs` a ctypes double."""
    fn = load().fa_probe_read_bandwidth
    if fn.argtypes is None:
        fn.argtypes = [_vp, ctypes.c_size_t, _int, _vp, ctypes.POINTER(ctypes.c_double)]
        fn.restype = _int
    return fn(buf, nbytes, iters, stream, ctypes.byref(gbs))


def probe_read_bandwidth(t, iters: int = 5) -> float:
    """HBM read rate (GB/s) measured by reading the CUDA tensor `t` (contiguous, far
    larger than L2; its first multiple of 16 bytes is read, nothing is written)."""
    _check("t", t, t.dtype)
    nbytes = t.numel() * t.element_size() // 16 * 16
    gbs = ctypes.c_double(0.0)
    with torch.cuda.device(t.device):
        rc = fa_probe_read_bandwidth(t.data_ptr(), nbytes, int(iters), _stream(t, None), gbs)
    if rc != FA_OK:
        raise FaError(rc, "fa_probe_read_bandwidth")
    return gbs.value


def probe_unit_rates(iters: int = 2048, stream=None) -> dict:
    """Measured per-SM rates on the current device: dense bf16 MMA FLOPs per SM clock
    at M = 128 with N = 256 and N = 64, and MUFU ex2 results per SM clock."""
    rates = (ctypes.c_double * 3)()
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    rc = fa_probe_unit_rates(rates, int(iters), stream)
    if rc != FA_OK:
        raise FaError(rc, "fa_probe_unit_rates")
    return {"mma_bf16_n256_flop_per_clk": rates[0], "mma_bf16_n64_flop_per_clk": rates[1],
            "ex2_per_clk": rates[2]}


def fa_fwd_workspace_bytes(B, H, N, d, causal, kv_chunk=0) -> int:
    fn = load().fa_fwd_workspace_bytes
    if fn.argtypes is None:
        fn.argtypes = [_int] * 6
        fn.restype = ctypes.c_size_t
    return fn(B, H, N, d, int(bool(causal)), kv_chunk)


def fa_fwd_split_segments(B, H, N, d, causal, num_sms, out=None, cap=0) -> int:
    """Raw call: fills `out` (ctypes int array of 7 * cap) and returns the count."""
    fn = load().fa_fwd_split_segments
    if fn.argtypes is None:
        fn.argtypes = [_int] * 6 + [_vp, _int]
        fn.restype = _int
    return fn(B, H, N, d, int(bool(causal)), num_sms, out, cap)


def fwd_split_segments(B, H, N, d, causal, num_sms):
    """The balanced cut of fa_fwd_ws (kv_chunk = 0) for num_sms SMs, as a list of
    (head, row block, first K/V tile, K/V tiles, part, parts, CTA) tuples ([]: no
    such cut).  Host only."""
    n = fa_fwd_split_segments(B, H, N, d, causal, num_sms)
    if n < 0:
        raise FaError(n, "fa_fwd_split_segments")
    if n == 0:
        return []
    buf = (ctypes.c_int * (7 * n))()
    fa_fwd_split_segments(B, H, N, d, causal, num_sms, ctypes.cast(buf, _vp), n)
    return [tuple(buf[7 * i:7 * i + 7]) for i in range(n)]


def fa_fwd_ws(q, k, v, o, lse, B, H, Hkv, N, d, causal, scale, kv_chunk, workspace,
              workspace_bytes, stream) -> int:
    fn = load().fa_fwd_ws
    if fn.argtypes is None:
        fn.argtypes = [_vp] * 5 + [_int] * 6 + [ctypes.c_float, _int, _vp, ctypes.c_size_t, _vp]
        fn.restype = _int
    return fn(q, k, v, o, lse, B, H, Hkv, N, d, int(bool(causal)), scale, kv_chunk, workspace,
              workspace_bytes, stream)


def fa_fwd_gqa(q, k, v, o, lse, B, H, Hkv, N, d, causal, scale, stream) -> int:
    return load().fa_fwd_gqa(q, k, v, o, lse, B, H, Hkv, N, d, int(bool(causal)), scale, stream)


def fa_bwd_gqa(q, k, v, o, lse, dout, dq, dk, dv, B, H, Hkv, N, d, causal, scale, workspace,
               workspace_bytes, stream) -> int:
    return load().fa_bwd_gqa(q, k, v, o, lse, dout, dq, dk, dv, B, H, Hkv, N, d, int(bool(causal)),
                             scale, workspace, workspace_bytes, stream)


def fa_fwd_varlen(q, k, v, o, lse, cu_seqlens, B, H, Hkv, total_tokens, max_seqlen, d, causal,
                  scale, stream) -> int:
    return load().fa_fwd_varlen(q, k, v, o, lse, cu_seqlens, B, H, Hkv, total_tokens, max_seqlen,
                                d, int(bool(causal)), scale, stream)


def fa_bwd_varlen(q, k, v, o, lse, dout, dq, dk, dv, cu_seqlens, B, H, Hkv, total_tokens,
                  max_seqlen, d, causal, scale, workspace, workspace_bytes, stream) -> int:
    return load().fa_bwd_varlen(q, k, v, o, lse, dout, dq, dk, dv, cu_seqlens, B, H, Hkv,
                                total_tokens, max_seqlen, d, int(bool(causal)), scale, workspace,
                                workspace_bytes, stream)


def fa_quantize_fp8_workspace_bytes(BH, N, d) -> int:
    return load().fa_quantize_fp8_workspace_bytes(BH, N, d)


def fa_quantize_fp8(x, codes, descale, BH, N, d, block_rows, signs, transpose, workspace,
                    workspace_bytes, stream) -> int:
    return load().fa_quantize_fp8(x, codes, descale, BH, N, d, block_rows, signs,
                                  int(bool(transpose)), workspace, workspace_bytes, stream)


def fa_fwd_fp8(q8, k8, vt8, q_descale, k_descale, v_descale, o, lse, B, H, Hkv, N, d, causal,
               scale, stream) -> int:
    return load().fa_fwd_fp8(q8, k8, vt8, q_descale, k_descale, v_descale, o, lse, B, H, Hkv, N,
                             d, int(bool(causal)), scale, stream)


def fa_decode(q, k, v, o, lse, B, H, Hkv, Nq, Nk, d, scale, num_splits, workspace,
              workspace_bytes, stream) -> int:
    return load().fa_decode(q, k, v, o, lse, B, H, Hkv, Nq, Nk, d, scale, num_splits, workspace,
                            workspace_bytes, stream)


def fa_decode_num_splits(B, H, Hkv, Nq, Nk, d, num_splits=0) -> int:
    return load().fa_decode_num_splits(B, H, Hkv, Nq, Nk, d, num_splits)


def fa_decode_uses_tensor_cores(H, Hkv, Nq, d, paged=0) -> int:
    return load().fa_decode_uses_tensor_cores(H, Hkv, Nq, d, int(paged))


def fa_decode_workspace_bytes(B, H, Hkv, Nq, Nk, d, num_splits=0) -> int:
    return load().fa_decode_workspace_bytes(B, H, Hkv, Nq, Nk, d, num_splits)


def fa_decode_paged(q, k_cache, v_cache, block_table, seq_lens, o, lse, B, H, Hkv, Nq, d,
                    page_size, max_pages, num_pages, scale, num_splits, workspace,
                    workspace_bytes, stream) -> int:
    return load().fa_decode_paged(q, k_cache, v_cache, block_table, seq_lens, o, lse, B, H, Hkv,
                                  Nq, d, page_size, max_pages, num_pages, scale, num_splits,
                                  workspace, workspace_bytes, stream)


def fa_decode_paged_num_splits(B, H, Hkv, Nq, d, page_size, max_pages, num_splits=0) -> int:
    return load().fa_decode_paged_num_splits(B, H, Hkv, Nq, d, page_size, max_pages, num_splits)


def fa_decode_paged_workspace_bytes(B, H, Hkv, Nq, d, page_size, max_pages, num_splits=0) -> int:
    return load().fa_decode_paged_workspace_bytes(B, H, Hkv, Nq, d, page_size, max_pages,
                                                  num_splits)


def fa_append_paged_fp8(k, v, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens,
                        B, T, Hkv, d, page_size, max_pages, num_pages, scale_group, k_stride,
                        v_stride, stream) -> int:
    return load().fa_append_paged_fp8(k, v, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                                      cu_seqlens, B, T, Hkv, d, page_size, max_pages, num_pages,
                                      scale_group, k_stride, v_stride, stream)


def fa_decode_paged_fp8_workspace_bytes(B, H, Hkv, Nq, d, page_size, max_pages) -> int:
    return load().fa_decode_paged_fp8_workspace_bytes(B, H, Hkv, Nq, d, page_size, max_pages)


def fa_decode_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, o, lse, B, H,
                        Hkv, Nq, d, page_size, max_pages, num_pages, scale_group, causal, scale,
                        workspace, workspace_bytes, stream) -> int:
    return load().fa_decode_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, o,
                                      lse, B, H, Hkv, Nq, d, page_size, max_pages, num_pages,
                                      scale_group, int(bool(causal)), scale, workspace,
                                      workspace_bytes, stream)


def fa_free_pages(block_table, seq_lens, pages, count, B, max_pages, page_size, num_pages,
                  stream) -> int:
    return load().fa_free_pages(block_table, seq_lens, pages, count, B, max_pages, page_size,
                                num_pages, stream)


def fa_fork_pages(block_table, seq_lens, parents, fresh, rows, lens, src, dst, B, n, max_pages,
                  page_size, num_pages, stream) -> int:
    return load().fa_fork_pages(block_table, seq_lens, parents, fresh, rows, lens, src, dst, B, n,
                                max_pages, page_size, num_pages, stream)


def fa_compact_pages(block_table, seq_lens, new_table, src, dst, counts, B, max_pages, page_size,
                     num_pages, stream) -> int:
    return load().fa_compact_pages(block_table, seq_lens, new_table, src, dst, counts, B, max_pages,
                                   page_size, num_pages, stream)


def fa_copy_pages(caches, page_bytes, n_caches, num_pages, src, dst, n_pairs, count, stream) -> int:
    """Raw call; `caches` and `page_bytes` are ctypes arrays of void* and size_t (host)."""
    return load().fa_copy_pages(caches, page_bytes, n_caches, num_pages, src, dst, n_pairs, count,
                                stream)


def fa_decode_paged_tree_workspace_bytes(B, H, Hkv, Nq, Nt, d, page_size, max_pages) -> int:
    return load().fa_decode_paged_tree_workspace_bytes(B, H, Hkv, Nq, Nt, d, page_size, max_pages)


def fa_decode_paged_tree(q, k_cache, v_cache, block_table, seq_lens, parents, o, lse, B, H, Hkv, Nq, Nt,
                         d, page_size, max_pages, num_pages, scale, workspace, workspace_bytes,
                         stream) -> int:
    return load().fa_decode_paged_tree(q, k_cache, v_cache, block_table, seq_lens, parents, o, lse, B, H,
                                       Hkv, Nq, Nt, d, page_size, max_pages, num_pages, scale, workspace,
                                       workspace_bytes, stream)


def fa_verify_tree(tokens, parents, target_probs, draft_probs, uniform, path, new_tokens, count, B, Nt, V,
                   bf16, replacement, stream) -> int:
    return load().fa_verify_tree(tokens, parents, target_probs, draft_probs, uniform, path, new_tokens,
                                 count, B, Nt, V, int(bool(bf16)), int(bool(replacement)), stream)


def fa_keep_path(caches, n_caches, block_table, seq_lens, path, count, lens, B, Nt, Hkv, d, page_size,
                 max_pages, num_pages, stream) -> int:
    """Raw call; `caches` is a ctypes array of void* (host)."""
    return load().fa_keep_path(caches, n_caches, block_table, seq_lens, path, count, lens, B, Nt, Hkv, d,
                               page_size, max_pages, num_pages, stream)


def fa_status_string(status: int) -> str:
    return load().fa_status_string(status).decode()


def fa_device_status(stream=None) -> int:
    return load().fa_device_status(stream)


# ------------------------------------------------------------ tensor wrappers

def _check(name, t, dtype, shape=None, dev=None):
    """Argument checks before any launch: a contiguous CUDA tensor of `dtype` (and
    `shape`) on device `dev` (a torch.device or an ordinal), the first tensor's device:
    the kernels dereference every pointer on that one GPU."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev is not None and t.get_device() != (dev if isinstance(dev, int) else dev.index):
        raise ValueError(f"{name} is on {t.device}, the call's first tensor on {dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


# The current stream's handle: torch's raw getter where it has one (a plain integer,
# no Stream object is built), else the public call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t, stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(t.get_device())
        return torch.cuda.current_stream(t.device).cuda_stream
    if not isinstance(stream, torch.cuda.Stream):
        return int(stream)
    _same_device(t, stream)
    return stream.cuda_stream


def _same_device(t, stream):
    if isinstance(t, torch.Tensor) and t.is_cuda and stream.device_index != t.get_device():
        raise ValueError(f"stream is on cuda:{stream.device_index}, the tensors on {t.device}")


def _under(stream, t, fn, *args):
    """fn(*args), a call on GPU tensors like `t`, with `stream` (a torch stream or a handle) as
    the current one: what the call allocates belongs to the stream that its kernels run on, so
    scratch that is released on return is handed out again only behind them.  Results it made
    are marked as in use on the caller's stream too."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return fn(*args)  # which refuses it
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), t.device)
    _same_device(t, stream)
    caller = torch.cuda.current_stream(t.device)
    with torch.cuda.stream(stream):
        result = fn(*args)
    for r in result:
        if not any(r is a for a in args):
            r.record_stream(caller)
    return result


_SAME_DEVICE = contextlib.nullcontext()


def _device(index: int):
    """The device context for a call on GPU `index`: a no-op when it is already
    current (the common case), else torch.cuda.device(index)."""
    return _SAME_DEVICE if torch.cuda.current_device() == index else torch.cuda.device(index)


_SIZE_MEMO: dict = {}


def _memo(fn, *args):
    """fn(*args) for the workspace-size queries, remembered per argument tuple and
    current device (the answers depend only on them and the device's SM count)."""
    key = (fn, torch.cuda.current_device(), args)
    r = _SIZE_MEMO.get(key)
    if r is None:
        if len(_SIZE_MEMO) > 4096:
            _SIZE_MEMO.clear()
        r = _SIZE_MEMO[key] = fn(*args)
    return r


def _kv_heads(q, k, v):
    """Key/value head count of k, v [B, Hkv, N, d] next to q [B, H, N, d] (Hkv divides H)."""
    B, H, N, d = q.shape
    di = q.get_device()
    _check("k", k, torch.bfloat16, dev=di)
    if k.dim() != 4 or k.shape[0] != B or k.shape[2] != N or k.shape[3] != d or H % k.shape[1]:
        raise ValueError("k must be [B, Hkv, N, d] with Hkv dividing q's H")
    _check("v", v, torch.bfloat16, k.shape, dev=di)
    return k.shape[1]


def forward(q, k, v, causal=False, scale=None, out=None, lse=None, stream=None, kv_chunk=0,
            workspace=None):
    """O, L = attention(q, k, v); q bf16 CUDA [B,H,N,d], k/v [B,Hkv,N,d] (Hkv = H, or
    fewer heads shared by groups of query heads).  Returns (o, lse).

    When few long heads would leave SMs idle, the key ranges are cut over several
    CTAs and merged (fa_fwd_ws): kv_chunk = 0 lets the library decide, > 0 asks for
    chunks of about that many keys; the workspace that needs is allocated here
    unless given."""
    if stream is not None:
        return _under(stream, q, forward, q, k, v, causal, scale, out, lse, None, kv_chunk,
                      workspace)
    _check("q", q, torch.bfloat16)
    if q.dim() != 4:
        raise ValueError("q must be [B, H, N, d]")
    B, H, N, d = q.shape
    di = q.get_device()
    Hkv = _kv_heads(q, k, v)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    _check("out", out, torch.bfloat16, q.shape, dev=di)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check("lse", lse, torch.float32, (B, H, N), dev=di)
    with _device(di):
        need = _memo(fa_fwd_workspace_bytes, B, H, N, d, causal, int(kv_chunk))
        if need == 0:
            rc = fa_fwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                            lse.data_ptr(), B, H, Hkv, N, d, causal, scale, _stream(q, None))
            where = "fa_fwd_gqa"
        else:
            if workspace is None:
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            _check("workspace", workspace, torch.uint8, dev=q.device)
            rc = fa_fwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                           lse.data_ptr(), B, H, Hkv, N, d, causal, scale, int(kv_chunk),
                           workspace.data_ptr(), workspace.numel(), _stream(q, None))
            where = "fa_fwd_ws"
    if rc != FA_OK:
        raise FaError(rc, where)
    return out, lse


def backward(q, k, v, o, lse, do, causal=False, scale=None, dq=None, dk=None, dv=None,
             workspace=None, stream=None):
    """dQ, dK, dV (fp32) of attention(q, k, v) given dO; o and lse from forward().
    With fewer key/value heads (k, v [B,Hkv,N,d]) dK, dV are [B,Hkv,N,d] sums over
    each head's query group."""
    if stream is not None:
        return _under(stream, q, backward, q, k, v, o, lse, do, causal, scale, dq, dk, dv,
                      workspace)
    _check("q", q, torch.bfloat16)
    if q.dim() != 4:
        raise ValueError("q must be [B, H, N, d]")
    B, H, N, d = q.shape
    Hkv = _kv_heads(q, k, v)
    for name, t in (("o", o), ("do", do)):
        _check(name, t, torch.bfloat16, q.shape, dev=q.device)
    _check("lse", lse, torch.float32, (B, H, N), dev=q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    grads = []
    for name, t, shape in (("dq", dq, q.shape), ("dk", dk, k.shape), ("dv", dv, k.shape)):
        if t is None:
            t = torch.empty(shape, dtype=torch.float32, device=q.device)
        _check(name, t, torch.float32, shape, dev=q.device)
        grads.append(t)
    need = fa_bwd_workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check("workspace", workspace, torch.uint8, dev=q.device)
    with torch.cuda.device(q.device):
        rc = fa_bwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                        do.data_ptr(), grads[0].data_ptr(), grads[1].data_ptr(),
                        grads[2].data_ptr(), B, H, Hkv, N, d, causal, scale, workspace.data_ptr(),
                        workspace.numel(), _stream(q, None))
    if rc != FA_OK:
        raise FaError(rc, "fa_bwd_gqa")
    return tuple(grads)


def decode(q, k, v, scale=None, num_splits=0, out=None, lse=None, workspace=None, stream=None):
    """Decode attention: q bf16 CUDA [B,H,Nq,d] against the cache k, v [B,Hkv,Nk,d]
    (Hkv divides H; no mask), the key range split over CTAs and merged by LSE.
    Returns (o, lse)."""
    if stream is not None:
        return _under(stream, q, decode, q, k, v, scale, num_splits, out, lse, workspace)
    _check("q", q, torch.bfloat16)
    if q.dim() != 4:
        raise ValueError("q must be [B, H, Nq, d]")
    B, H, Nq, d = q.shape
    di = q.get_device()
    _check("k", k, torch.bfloat16, dev=di)
    if k.dim() != 4 or k.shape[0] != B or k.shape[3] != d or H % k.shape[1]:
        raise ValueError("k must be [B, Hkv, Nk, d] with q's B and d, Hkv dividing H")
    Hkv, Nk = k.shape[1], k.shape[2]
    _check("v", v, torch.bfloat16, k.shape, dev=di)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    _check("out", out, torch.bfloat16, q.shape, dev=di)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    _check("lse", lse, torch.float32, (B, H, Nq), dev=di)
    with _device(di):
        need = _memo(fa_decode_workspace_bytes, B, H, Hkv, Nq, Nk, d, num_splits)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        if workspace is not None:
            _check("workspace", workspace, torch.uint8, dev=di)
        ws_ptr = workspace.data_ptr() if workspace is not None else None
        ws_len = workspace.numel() if workspace is not None else 0
        rc = fa_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                       B, H, Hkv, Nq, Nk, d, scale, num_splits, ws_ptr, ws_len, _stream(q, None))
    if rc != FA_OK:
        raise FaError(rc, "fa_decode")
    return out, lse


def decode_paged(q, k_cache, v_cache, block_table, seq_lens, scale=None, num_splits=0, out=None,
                 lse=None, workspace=None, stream=None):
    """Decode against a paged cache: q bf16 [B,H,Nq,d]; k_cache, v_cache bf16
    [num_pages, Hkv, page_size, d] (Hkv divides H); block_table int32 [B, max_pages];
    seq_lens int32 [B] (all CUDA).  Returns (o, lse)."""
    if stream is not None:
        return _under(stream, q, decode_paged, q, k_cache, v_cache, block_table, seq_lens, scale,
                      num_splits, out, lse, workspace)
    _check("q", q, torch.bfloat16)
    if q.dim() != 4:
        raise ValueError("q must be [B, H, Nq, d]")
    B, H, Nq, d = q.shape
    _check("k_cache", k_cache, torch.bfloat16, dev=q.device)
    if k_cache.dim() != 4 or H % k_cache.shape[1] or k_cache.shape[3] != d:
        raise ValueError("k_cache must be [num_pages, Hkv, page_size, d], Hkv dividing H")
    num_pages, Hkv, page_size, _ = k_cache.shape
    _check("v_cache", v_cache, torch.bfloat16, k_cache.shape, dev=q.device)
    _check("block_table", block_table, torch.int32, dev=q.device)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages]")
    max_pages = block_table.shape[1]
    _check("seq_lens", seq_lens, torch.int32, (B,), dev=q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    _check("out", out, torch.bfloat16, q.shape, dev=q.device)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    _check("lse", lse, torch.float32, (B, H, Nq), dev=q.device)
    with torch.cuda.device(q.device):
        need = fa_decode_paged_workspace_bytes(B, H, Hkv, Nq, d, page_size, max_pages, num_splits)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        if workspace is not None:
            _check("workspace", workspace, torch.uint8, dev=q.device)
        ws_ptr = workspace.data_ptr() if workspace is not None else None
        ws_len = workspace.numel() if workspace is not None else 0
        rc = fa_decode_paged(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                             block_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(),
                             lse.data_ptr(), B, H, Hkv, Nq, d, page_size, max_pages, num_pages,
                             scale, num_splits, ws_ptr, ws_len, _stream(q, None))
    if rc != FA_OK:
        raise FaError(rc, "fa_decode_paged")
    return out, lse


def forward_varlen(q, k, v, cu_seqlens, max_seqlen, causal=False, scale=None, out=None, lse=None,
                   stream=None):
    """Packed variable-length forward: q bf16 CUDA [T,H,d], k/v [T,Hkv,d], cu_seqlens
    int32 CUDA [B+1] (sequence b = tokens cu[b]..cu[b+1]-1, each <= max_seqlen).
    Returns (o [T,H,d], lse [H,T])."""
    if stream is not None:
        return _under(stream, q, forward_varlen, q, k, v, cu_seqlens, max_seqlen, causal, scale,
                      out, lse)
    _check("q", q, torch.bfloat16)
    if q.dim() != 3:
        raise ValueError("q must be [T, H, d]")
    T, H, d = q.shape
    _check("k", k, torch.bfloat16, dev=q.device)
    if k.dim() != 3 or k.shape[0] != T or k.shape[2] != d or H % k.shape[1]:
        raise ValueError("k must be [T, Hkv, d] with Hkv dividing H")
    Hkv = k.shape[1]
    _check("v", v, torch.bfloat16, k.shape, dev=q.device)
    _check("cu_seqlens", cu_seqlens, torch.int32, dev=q.device)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be [B + 1]")
    B = cu_seqlens.numel() - 1
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    _check("out", out, torch.bfloat16, q.shape, dev=q.device)
    if lse is None:
        lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
    _check("lse", lse, torch.float32, (H, T), dev=q.device)
    with torch.cuda.device(q.device):
        rc = fa_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                           cu_seqlens.data_ptr(), B, H, Hkv, T, int(max_seqlen), d, causal, scale,
                           _stream(q, None))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_varlen")
    return out, lse


def backward_varlen(q, k, v, o, lse, do, cu_seqlens, max_seqlen, causal=False, scale=None,
                    dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients of forward_varlen: q/o/do bf16 [T,H,d], k/v [T,Hkv,d], lse [H,T].
    Returns (dq [T,H,d], dk [T,Hkv,d], dv [T,Hkv,d]) fp32."""
    if stream is not None:
        return _under(stream, q, backward_varlen, q, k, v, o, lse, do, cu_seqlens, max_seqlen,
                      causal, scale, dq, dk, dv, workspace)
    _check("q", q, torch.bfloat16)
    if q.dim() != 3:
        raise ValueError("q must be [T, H, d]")
    T, H, d = q.shape
    _check("k", k, torch.bfloat16, dev=q.device)
    if k.dim() != 3 or k.shape[0] != T or k.shape[2] != d or H % k.shape[1]:
        raise ValueError("k must be [T, Hkv, d] with Hkv dividing H")
    Hkv = k.shape[1]
    _check("v", v, torch.bfloat16, k.shape, dev=q.device)
    for name, t in (("o", o), ("do", do)):
        _check(name, t, torch.bfloat16, q.shape, dev=q.device)
    _check("lse", lse, torch.float32, (H, T), dev=q.device)
    _check("cu_seqlens", cu_seqlens, torch.int32, dev=q.device)
    B = cu_seqlens.numel() - 1
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    grads = []
    for name, t, shape in (("dq", dq, q.shape), ("dk", dk, k.shape), ("dv", dv, k.shape)):
        if t is None:
            t = torch.zeros(shape, dtype=torch.float32, device=q.device)
        _check(name, t, torch.float32, shape, dev=q.device)
        grads.append(t)
    need = fa_bwd_workspace_bytes(B, H, int(max_seqlen), d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check("workspace", workspace, torch.uint8, dev=q.device)
    with torch.cuda.device(q.device):
        rc = fa_bwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                           do.data_ptr(), grads[0].data_ptr(), grads[1].data_ptr(),
                           grads[2].data_ptr(), cu_seqlens.data_ptr(), B, H, Hkv, T,
                           int(max_seqlen), d, causal, scale, workspace.data_ptr(),
                           workspace.numel(), _stream(q, None))
    if rc != FA_OK:
        raise FaError(rc, "fa_bwd_varlen")
    return tuple(grads)


def quantize_fp8(x, block_rows=128, signs=None, transpose=False, workspace=None, stream=None):
    """e4m3 block quantisation of x bf16 CUDA [..., N, d] (heads flattened).
    Returns (codes uint8 [..., N, d] or [..., d, Np], descale fp32 [..., n_blocks])."""
    if stream is not None:
        return _under(stream, x, quantize_fp8, x, block_rows, signs, transpose, workspace)
    _check("x", x, torch.bfloat16)
    if x.dim() < 2:
        raise ValueError("x must be [..., N, d]")
    *lead, N, d = x.shape
    BH = int(math.prod(lead)) if lead else 1
    Np = (N + 15) // 16 * 16
    codes = torch.empty((*lead, d, Np) if transpose else x.shape, dtype=torch.uint8, device=x.device)
    nb = 1 if block_rows == 0 else (N + block_rows - 1) // block_rows
    descale = torch.empty((*lead, nb), dtype=torch.float32, device=x.device)
    if signs is not None:
        _check("signs", signs, torch.float32, (d,), dev=x.device)
    need = fa_quantize_fp8_workspace_bytes(BH, N, d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    _check("workspace", workspace, torch.uint8, dev=x.device)
    with torch.cuda.device(x.device):
        rc = fa_quantize_fp8(x.data_ptr(), codes.data_ptr(), descale.data_ptr(), BH, N, d,
                             int(block_rows), None if signs is None else signs.data_ptr(),
                             transpose, workspace.data_ptr(), workspace.numel(), _stream(x, None))
    if rc != FA_OK:
        raise FaError(rc, "fa_quantize_fp8")
    return codes, descale


def forward_fp8(q8, k8, vt8, q_descale, k_descale, v_descale, causal=False, scale=None, out=None,
                lse=None, stream=None):
    """Attention on e4m3 inputs: q8 uint8 CUDA [B,H,N,d], k8 [B,Hkv,N,d], vt8 [B,Hkv,d,Np],
    q/k descales [B,H|Hkv,ceil(N/128)], v descale [B,Hkv,1].  Returns (o bf16, lse fp32)."""
    if stream is not None:
        return _under(stream, q8, forward_fp8, q8, k8, vt8, q_descale, k_descale, v_descale, causal,
                      scale, out, lse)
    _check("q8", q8, torch.uint8)
    if q8.dim() != 4:
        raise ValueError("q8 must be [B, H, N, d]")
    B, H, N, d = q8.shape
    _check("k8", k8, torch.uint8, dev=q8.device)
    if k8.dim() != 4 or k8.shape[0] != B or k8.shape[2] != N or k8.shape[3] != d or H % k8.shape[1]:
        raise ValueError("k8 must be [B, Hkv, N, d] with Hkv dividing H")
    Hkv = k8.shape[1]
    Np = (N + 15) // 16 * 16
    _check("vt8", vt8, torch.uint8, (B, Hkv, d, Np), dev=q8.device)
    nb = (N + 127) // 128
    _check("q_descale", q_descale, torch.float32, (B, H, nb), dev=q8.device)
    _check("k_descale", k_descale, torch.float32, (B, Hkv, nb), dev=q8.device)
    _check("v_descale", v_descale, torch.float32, (B, Hkv, 1), dev=q8.device)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q8.device)
    _check("out", out, torch.bfloat16, (B, H, N, d), dev=q8.device)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q8.device)
    _check("lse", lse, torch.float32, (B, H, N), dev=q8.device)
    with torch.cuda.device(q8.device):
        rc = fa_fwd_fp8(q8.data_ptr(), k8.data_ptr(), vt8.data_ptr(), q_descale.data_ptr(),
                        k_descale.data_ptr(), v_descale.data_ptr(), out.data_ptr(), lse.data_ptr(),
                        B, H, Hkv, N, d, causal, scale, _stream(q8, None))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_fp8")
    return out, lse


# The calls on a paged cache are made many times per decode step on kernels of a few
# microseconds, so the extension makes them: it answers with the outputs, with a status, or
# with None when an argument is not as expected.  What follows it here names the argument
# that is wrong (and serves the calls the extension leaves alone, tensor subclasses).  The int32
# outputs of one call of the extension are parts of one allocation, which any of them keeps.

def _raw(stream, t):
    return None if stream is None else _stream(t, stream)


def _ok(status, where):
    if status != FA_OK:
        raise FaError(status, where)


def _cache8(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, di):
    """Checks of a paged e4m3 cache and its table on device `di`; returns (B, num_pages, Hkv,
    page_size, d, max_pages, scale_group)."""
    _check("k_cache", k_cache, torch.uint8, dev=di)
    if k_cache.dim() != 4 or 0 in k_cache.shape:
        raise ValueError("k_cache must be [num_pages, Hkv, page_size, d]")
    num_pages, Hkv, page_size, d = k_cache.shape
    _check("v_cache", v_cache, torch.uint8, k_cache.shape, dev=di)
    _check("k_scale", k_scale, torch.float32, dev=di)
    groups = k_scale.shape[2] if k_scale.dim() == 3 else 0
    if groups < 1 or page_size % groups or k_scale.shape[:2] != k_cache.shape[:2]:
        raise ValueError("k_scale must be [num_pages, Hkv, page_size / group]")
    _check("v_scale", v_scale, torch.float32, k_scale.shape, dev=di)
    _check("block_table", block_table, torch.int32, dev=di)
    if block_table.dim() != 2 or block_table.shape[1] < 1:
        raise ValueError("block_table must be [B, max_pages]")
    B, max_pages = block_table.shape
    _check("seq_lens", seq_lens, torch.int32, (B,), dev=di)
    return B, num_pages, Hkv, page_size, d, max_pages, page_size // groups


def _check_rows(name, t, dtype, shape, di):
    """A CUDA tensor [T, Hkv, d] whose rows of Hkv * d elements are contiguous, at any stride."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != di:
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{di}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or t.shape[1:] != shape or t.shape[0] < 1:
        raise ValueError(f"{name} must be [T, {shape[0]}, {shape[1]}], T >= 1")
    if t.stride(2) != 1 or (t.stride(1) != shape[1] and shape[0] > 1):
        raise ValueError(f"{name}'s rows [Hkv, d] must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), shape[0] * shape[1])


def append_paged_fp8(k, v, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                     cu_seqlens=None, stream=None):
    """Store new tokens in a paged e4m3 cache, behind the seq_lens[b] tokens that sequence b
    holds: k, v bf16 CUDA [T, Hkv, d] (rows contiguous, any row stride that is a multiple of
    8), rows cu_seqlens[b] .. cu_seqlens[b+1]-1 belonging to sequence b (int32 [B+1]; None:
    one new token each).  The cache is uint8 codes [num_pages, Hkv, page_size, d] and fp32
    scales [num_pages, Hkv, page_size / group], group at most 128, for k and for v, changed in
    place; seq_lens is not changed.  Returns None."""
    r = native().append_paged_fp8(k, v, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                                  cu_seqlens, _raw(stream, k))
    if r is not None:
        return _ok(r, "fa_append_paged_fp8")
    di = k_cache.get_device() if isinstance(k_cache, torch.Tensor) else -1
    B, num_pages, Hkv, page_size, d, max_pages, group = _cache8(k_cache, v_cache, k_scale, v_scale,
                                                                block_table, seq_lens, di)
    ks = _check_rows("k", k, torch.bfloat16, (Hkv, d), di)
    vs = _check_rows("v", v, torch.bfloat16, (Hkv, d), di)
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError("k and v must have the same number of rows")
    cu = None
    if cu_seqlens is not None:
        _check("cu_seqlens", cu_seqlens, torch.int32, (B + 1,), dev=di)
        cu = cu_seqlens.data_ptr()
    elif T != B:
        raise ValueError("without cu_seqlens, k and v hold one row per sequence")
    with _device(di):
        rc = fa_append_paged_fp8(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                 k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(),
                                 seq_lens.data_ptr(), cu, B, T, Hkv, d, page_size, max_pages,
                                 num_pages, group, ks, vs, _stream(k, stream))
    _ok(rc, "fa_append_paged_fp8")


def decode_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, causal=False,
                     scale=None, out=None, lse=None, workspace=None, stream=None):
    """Decode against a paged e4m3 cache: q bf16 CUDA [B,H,Nq,d]; k_cache, v_cache uint8 codes
    [num_pages, Hkv, page_size, d] (Hkv divides H) with scales fp32 [num_pages, Hkv, page_size /
    group], >= 0 and at most 2^120; block_table int32 [B, max_pages]; seq_lens int32 [B], 0
    allowed.  causal: the Nq queries are the sequence's last tokens, each sees the keys up to its
    own.  Rows that see no key get o = 0 and lse = -inf.  Returns (o, lse)."""
    r = native().decode_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, causal,
                                  scale, out, lse, workspace, _raw(stream, q))
    if r.__class__ is tuple:
        return r
    if r is not None:
        raise FaError(r, "fa_decode_paged_fp8")
    if stream is not None:
        return _under(stream, q, decode_paged_fp8, q, k_cache, v_cache, k_scale, v_scale, block_table,
                      seq_lens, causal, scale, out, lse, workspace)
    _check("q", q, torch.bfloat16)
    if q.dim() != 4:
        raise ValueError("q must be [B, H, Nq, d]")
    B, H, Nq, d = q.shape
    di = q.get_device()
    B2, num_pages, Hkv, page_size, d2, max_pages, group = _cache8(k_cache, v_cache, k_scale, v_scale,
                                                                  block_table, seq_lens, di)
    if B2 != B:
        raise ValueError("block_table must be [B, max_pages]")
    if d2 != d or H % Hkv:
        raise ValueError("k_cache must be [num_pages, Hkv, page_size, d], Hkv dividing H")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check("out", out, torch.bfloat16, q.shape, dev=di)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    else:
        _check("lse", lse, torch.float32, (B, H, Nq), dev=di)
    with _device(di):
        need = _memo(fa_decode_paged_fp8_workspace_bytes, B, H, Hkv, Nq, d, page_size, max_pages)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:
            _check("workspace", workspace, torch.uint8, dev=di)
        rc = fa_decode_paged_fp8(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                 k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(),
                                 seq_lens.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, Hkv, Nq,
                                 d, page_size, max_pages, num_pages, group, causal, scale,
                                 workspace.data_ptr(), workspace.numel(), _stream(q, None))
    _ok(rc, "fa_decode_paged_fp8")
    return out, lse


def _table(block_table, seq_lens):
    _check("block_table", block_table, torch.int32)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    _check("seq_lens", seq_lens, torch.int32, block_table.shape[:1], dev=block_table.get_device())
    return block_table.get_device(), *block_table.shape


def _int32(shape, like):
    return torch.empty(shape, dtype=torch.int32, device=like.device)


def free_pages(block_table, seq_lens, page_size, num_pages, stream=None):
    """The pages of a paged cache that no sequence uses: (pages int32 [num_pages], ascending,
    then -1; count int32 [1])."""
    r = native().free_pages(block_table, seq_lens, page_size, num_pages, _raw(stream, block_table))
    if r.__class__ is tuple:
        return r
    if r is not None:
        raise FaError(r, "fa_free_pages")
    if stream is not None:
        return _under(stream, block_table, free_pages, block_table, seq_lens, page_size, num_pages)
    di, B, max_pages = _table(block_table, seq_lens)
    pages, count = _int32(max(int(num_pages), 0), block_table), _int32(1, block_table)
    with _device(di):
        rc = fa_free_pages(block_table.data_ptr(), seq_lens.data_ptr(), pages.data_ptr(),
                           count.data_ptr(), B, max_pages, int(page_size), int(num_pages),
                           _stream(block_table, None))
    _ok(rc, "fa_free_pages")
    return pages, count


def fork_pages(block_table, seq_lens, parents, fresh, page_size, num_pages, stream=None):
    """Children of the sequences `parents` (int32 [n], rows of block_table): they share the
    parents' full pages, and child i takes page fresh[i] (int32 [n]) for a copy of a last page
    that is not full.  Returns (rows int32 [n, max_pages], lens [n], src [n], dst [n]): the
    children's table rows and lengths, and the pages to pass to copy_pages (-1: none)."""
    r = native().fork_pages(block_table, seq_lens, parents, fresh, page_size, num_pages,
                            _raw(stream, block_table))
    if r.__class__ is tuple:
        return r
    if r is not None:
        raise FaError(r, "fa_fork_pages")
    if stream is not None:
        return _under(stream, block_table, fork_pages, block_table, seq_lens, parents, fresh, page_size,
                      num_pages)
    di, B, max_pages = _table(block_table, seq_lens)
    _check("parents", parents, torch.int32, dev=di)
    if parents.dim() != 1:
        raise ValueError("parents must be [n]")
    _check("fresh", fresh, torch.int32, parents.shape, dev=di)
    n = parents.shape[0]
    rows, lens, src, dst = (_int32(s, block_table) for s in ((n, max_pages), n, n, n))
    with _device(di):
        rc = fa_fork_pages(block_table.data_ptr(), seq_lens.data_ptr(), parents.data_ptr(),
                           fresh.data_ptr(), rows.data_ptr(), lens.data_ptr(), src.data_ptr(),
                           dst.data_ptr(), B, n, max_pages, int(page_size), int(num_pages),
                           _stream(block_table, None))
    _ok(rc, "fa_fork_pages")
    return rows, lens, src, dst


def compact_pages(block_table, seq_lens, page_size, num_pages, stream=None):
    """Plan that packs the n pages in use into pages 0 .. n-1: (table int32 [B, max_pages] after
    the moves, src, dst int32 [max(1, num_pages // 2)] ending in -1, counts int32 [2] = n and
    the number of moves).  copy_pages(caches, src, dst, count=counts[1:]) makes the moves."""
    r = native().compact_pages(block_table, seq_lens, page_size, num_pages, _raw(stream, block_table))
    if r.__class__ is tuple:
        return r
    if r is not None:
        raise FaError(r, "fa_compact_pages")
    if stream is not None:
        return _under(stream, block_table, compact_pages, block_table, seq_lens, page_size, num_pages)
    di, B, max_pages = _table(block_table, seq_lens)
    cap = max(1, int(num_pages) // 2)
    table, src, dst, counts = (_int32(s, block_table) for s in ((B, max_pages), cap, cap, 2))
    with _device(di):
        rc = fa_compact_pages(block_table.data_ptr(), seq_lens.data_ptr(), table.data_ptr(),
                              src.data_ptr(), dst.data_ptr(), counts.data_ptr(), B, max_pages,
                              int(page_size), int(num_pages), _stream(block_table, None))
    _ok(rc, "fa_compact_pages")
    return table, src, dst, counts


FA_MAX_COPY_CACHES = 128


def copy_pages(caches, src, dst, count=None, stream=None):
    """Copy page src[i] of every tensor of `caches` (contiguous CUDA tensors, their first
    dimension num_pages: codes and scales, any number of layers up to 128 tensors) onto its page
    dst[i], for every pair of int32 [n] src, dst with src[i] != -1; with `count` (int32 [1]) only
    the first count pairs.  No page may be a destination twice, or destination and source."""
    caches = caches if isinstance(caches, list) else list(caches)
    r = native().copy_pages(caches, src, dst, count, _raw(stream, src))
    if r is not None:
        return _ok(r, "fa_copy_pages")
    if not 1 <= len(caches) <= FA_MAX_COPY_CACHES:
        raise ValueError(f"caches must be 1 to {FA_MAX_COPY_CACHES} tensors")
    di = src.get_device() if isinstance(src, torch.Tensor) else -1
    _check("src", src, torch.int32)
    if src.dim() != 1:
        raise ValueError("src must be [n]")
    _check("dst", dst, torch.int32, src.shape, dev=di)
    if count is not None:
        _check("count", count, torch.int32, (1,), dev=di)
    num_pages = caches[0].shape[0] if isinstance(caches[0], torch.Tensor) and caches[0].dim() else 0
    ptrs = (_vp * len(caches))()
    sizes = (ctypes.c_size_t * len(caches))()
    for i, t in enumerate(caches):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"caches[{i}] must be a CUDA tensor")
        _check(f"caches[{i}]", t, t.dtype, dev=di)
        if t.dim() < 2 or t.shape[0] != num_pages or not t.numel():
            raise ValueError(f"caches[{i}] must be [num_pages, ...] like the first")
        ptrs[i] = t.data_ptr()
        sizes[i] = t.numel() // num_pages * t.element_size()
    with _device(di):
        rc = fa_copy_pages(ptrs, sizes, len(caches), num_pages, src.data_ptr(), dst.data_ptr(),
                           src.shape[0], None if count is None else count.data_ptr(),
                           _stream(src, stream))
    _ok(rc, "fa_copy_pages")


def _cache16(k_cache, v_cache, block_table, seq_lens, di):
    """Checks of a paged bf16 cache and its table on device `di`; returns (B, num_pages, Hkv,
    page_size, d, max_pages)."""
    _check("k_cache", k_cache, torch.bfloat16, dev=di)
    if k_cache.dim() != 4 or 0 in k_cache.shape:
        raise ValueError("k_cache must be [num_pages, Hkv, page_size, d]")
    num_pages, Hkv, page_size, d = k_cache.shape
    _check("v_cache", v_cache, torch.bfloat16, k_cache.shape, dev=di)
    _check("block_table", block_table, torch.int32, dev=di)
    if block_table.dim() != 2 or block_table.shape[1] < 1:
        raise ValueError("block_table must be [B, max_pages]")
    B, max_pages = block_table.shape
    _check("seq_lens", seq_lens, torch.int32, (B,), dev=di)
    return B, num_pages, Hkv, page_size, d, max_pages


def decode_paged_tree(q, k_cache, v_cache, block_table, seq_lens, parents=None, scale=None, out=None,
                      lse=None, workspace=None, stream=None):
    """Attention of drafted tokens against a paged bf16 cache: q bf16 CUDA [B,H,Nq,d], the queries
    of the last Nq of each sequence's Nt drafted tokens, whose keys and values lie in k_cache,
    v_cache bf16 [num_pages, Hkv, page_size, d] (Hkv divides H) behind the sequence's seq_lens[b]
    tokens (int32 [B], 0 allowed), through block_table int32 [B, max_pages].  parents int32 [B, Nt]:
    the number of an earlier drafted token, -1 for one without a parent among them, below -1 where
    there is none; None: Nt = Nq tokens drafted in a row.  A query sees the seq_lens[b] tokens,
    itself and its ancestors; where there is no token o = 0 and lse = -inf.  Returns (o, lse)."""
    r = native().decode_paged_tree(q, k_cache, v_cache, block_table, seq_lens, parents, scale, out, lse,
                                   workspace, _raw(stream, q))
    if r.__class__ is tuple:
        return r
    if r is not None:
        raise FaError(r, "fa_decode_paged_tree")
    if stream is not None:
        return _under(stream, q, decode_paged_tree, q, k_cache, v_cache, block_table, seq_lens, parents,
                      scale, out, lse, workspace)
    _check("q", q, torch.bfloat16)
    if q.dim() != 4:
        raise ValueError("q must be [B, H, Nq, d]")
    B, H, Nq, d = q.shape
    di = q.get_device()
    B2, num_pages, Hkv, page_size, d2, max_pages = _cache16(k_cache, v_cache, block_table, seq_lens, di)
    if B2 != B:
        raise ValueError("block_table must be [B, max_pages]")
    if d2 != d or H % Hkv:
        raise ValueError("k_cache must be [num_pages, Hkv, page_size, d], Hkv dividing H")
    Nt = Nq
    if parents is not None:
        _check("parents", parents, torch.int32, dev=di)
        if parents.dim() != 2 or parents.shape[0] != B or parents.shape[1] < Nq:
            raise ValueError("parents must be [B, Nt] with Nt >= Nq")
        Nt = parents.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check("out", out, torch.bfloat16, q.shape, dev=di)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    else:
        _check("lse", lse, torch.float32, (B, H, Nq), dev=di)
    with _device(di):
        need = _memo(fa_decode_paged_tree_workspace_bytes, B, H, Hkv, Nq, Nt, d, page_size, max_pages)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:
            _check("workspace", workspace, torch.uint8, dev=di)
        rc = fa_decode_paged_tree(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                  block_table.data_ptr(), seq_lens.data_ptr(),
                                  None if parents is None else parents.data_ptr(), out.data_ptr(),
                                  lse.data_ptr(), B, H, Hkv, Nq, Nt, d, page_size, max_pages, num_pages,
                                  scale, workspace.data_ptr(), workspace.numel(), _stream(q, None))
    _ok(rc, "fa_decode_paged_tree")
    return out, lse


def verify_tree(tokens, parents, target_probs, draft_probs, uniform, replacement=True, stream=None):
    """Verification of drafted tokens: which of each sequence's tree are accepted, and one token more,
    distributed as the target's own samples.  tokens int32 CUDA [B, Nt], node 0 standing for the
    last certain token, the others drafted; parents int32 [B, Nt]: -1 for node 0, an earlier node's
    number for the others, below -1 where there is no node (None: a chain); target_probs [B, Nt, V]
    fp32 or bf16: the target's probabilities of the token after each node; draft_probs, alike: those
    that each node's children were drawn from (independently, or with replacement=False one after
    another without repetition), or None where drafts were not drawn; uniform fp32 [B, Nt] in [0, 1).
    Returns int32 (path [B, Nt], new_tokens [B, Nt], count [B]): the accepted nodes from node 0 on,
    the accepted tokens and the last one, each followed by -1, and how many there are of each."""
    r = native().verify_tree(tokens, parents, target_probs, draft_probs, uniform, replacement,
                             _raw(stream, tokens))
    if r.__class__ is tuple:
        return r
    if r is not None:
        raise FaError(r, "fa_verify_tree")
    if stream is not None:
        return _under(stream, tokens, verify_tree, tokens, parents, target_probs, draft_probs, uniform,
                      replacement)
    _check("tokens", tokens, torch.int32)
    if tokens.dim() != 2:
        raise ValueError("tokens must be [B, Nt]")
    B, Nt = tokens.shape
    di = tokens.get_device()
    if parents is not None:
        _check("parents", parents, torch.int32, tokens.shape, dev=di)
    dtype = target_probs.dtype if isinstance(target_probs, torch.Tensor) else None
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("target_probs must be a float32 or bfloat16 CUDA tensor")
    _check("target_probs", target_probs, dtype, dev=di)
    if target_probs.dim() != 3 or target_probs.shape[:2] != tokens.shape:
        raise ValueError("target_probs must be [B, Nt, V]")
    V = target_probs.shape[2]
    if draft_probs is not None:
        _check("draft_probs", draft_probs, dtype, target_probs.shape, dev=di)
    _check("uniform", uniform, torch.float32, tokens.shape, dev=di)
    path, new, count = (_int32(s, tokens) for s in ((B, Nt), (B, Nt), B))
    with _device(di):
        rc = fa_verify_tree(tokens.data_ptr(), None if parents is None else parents.data_ptr(),
                            target_probs.data_ptr(), None if draft_probs is None else draft_probs.data_ptr(),
                            uniform.data_ptr(), path.data_ptr(), new.data_ptr(), count.data_ptr(), B, Nt, V,
                            dtype == torch.bfloat16, replacement, _stream(tokens, None))
    _ok(rc, "fa_verify_tree")
    return path, new, count


def keep_path(caches, block_table, seq_lens, path, count, stream=None):
    """Keep the accepted nodes of drafted trees in a paged bf16 cache: behind sequence b's
    seq_lens[b] tokens (int32 CUDA [B]) the row of node path[b, i] (int32 [B, Nt], ascending) becomes
    row i for i < count[b] (int32 [B]), in every tensor of `caches` (bf16 [num_pages, Hkv, page_size,
    d], all of one shape, no two overlapping: keys and values of any number of layers, up to 128), through
    block_table int32 [B, max_pages].  Returns seq_lens + count, int32 [B]."""
    caches = caches if isinstance(caches, list) else list(caches)
    r = native().keep_path(caches, block_table, seq_lens, path, count, _raw(stream, block_table))
    if r.__class__ is tuple:
        return r[0]
    if r is not None:
        raise FaError(r, "fa_keep_path")
    if stream is not None:
        return _under(stream, block_table, lambda *a: (keep_path(*a),), caches, block_table, seq_lens, path,
                      count)[0]
    if not 1 <= len(caches) <= FA_MAX_COPY_CACHES:
        raise ValueError(f"caches must be 1 to {FA_MAX_COPY_CACHES} tensors")
    di, B, max_pages = _table(block_table, seq_lens)
    _check("caches[0]", caches[0], torch.bfloat16, dev=di)
    if caches[0].dim() != 4 or 0 in caches[0].shape:
        raise ValueError("caches[0] must be [num_pages, Hkv, page_size, d]")
    num_pages, Hkv, page_size, d = caches[0].shape
    ptrs = (_vp * len(caches))()
    for i, t in enumerate(caches):
        _check(f"caches[{i}]", t, torch.bfloat16, caches[0].shape, dev=di)
        ptrs[i] = t.data_ptr()
    _check("path", path, torch.int32, dev=di)
    if path.dim() != 2 or path.shape[0] != B:
        raise ValueError("path must be [B, Nt]")
    _check("count", count, torch.int32, (B,), dev=di)
    lens = _int32(B, block_table)
    with _device(di):
        rc = fa_keep_path(ptrs, len(caches), block_table.data_ptr(), seq_lens.data_ptr(), path.data_ptr(),
                          count.data_ptr(), lens.data_ptr(), B, path.shape[1], Hkv, d, page_size, max_pages,
                          num_pages, _stream(block_table, None))
    _ok(rc, "fa_keep_path")
    return lens
