"""Python binding of libmsa: ctypes declarations of include/msa.h and thin
wrappers with the same names that only marshal torch tensors into pointers.

Every step of the path runs in the CUDA library.  There is no CPU or PyTorch
fallback: if libmsa.so is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

from . import build as _build

MSA_OK, MSA_ERR_NULL, MSA_ERR_SHAPE, MSA_ERR_DTYPE, MSA_ERR_UNSUPPORTED, MSA_ERR_WORKSPACE, \
    MSA_ERR_CUDA = range(7)
MSA_KV_BF16, MSA_KV_FP8_E4M3 = 0, 1
MSA_SCALE_NONE, MSA_SCALE_SCALAR, MSA_SCALE_PER_TOKEN_HEAD = 0, 1, 2
MSA_DEV_BAD_PAGE, MSA_DEV_BAD_LEN, MSA_DEV_MALFORMED, MSA_DEV_BAD_TABLE, MSA_DEV_TIMEOUT = \
    1, 2, 4, 8, 16

EXPORTED = ("msa_index_score", "msa_topk_build_table", "msa_sparse_paged_attn", "msa_decode",
            "msa_kv_insert", "msa_sparse_mla_decode", "msa_sparse_mla_workspace_size",
            "msa_workspace_size", "msa_status_string", "msa_check_bounded_wait",
            "msa_tree_attn_workspace_size", "msa_tree_attn", "msa_attn_mass", "msa_evict_select",
            "msa_kv_compact", "msa_qk_rope_insert", "msa_prompt_attn_workspace_size",
            "msa_prompt_attn", "msa_page_fork", "msa_page_copy")
MSA_DEV_BAD_POS, MSA_DEV_NO_PAGES = 32, 64
MSA_CHECK_WAIT_TMEM, MSA_CHECK_WAIT_COPY = 1, 2


class MsaError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn}: {status_string(code)} (status {code})")
        self.code = code


class msa_batch(ctypes.Structure):
    _fields_ = [("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
                ("context_lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("bt_stride", ctypes.c_int32), ("num_reqs", ctypes.c_int32),
                ("num_rows", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_q_len", ctypes.c_int32),
                ("min_q_len", ctypes.c_int32)]


class msa_attn_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("num_rows", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("k_cache", ctypes.c_void_p),
                ("v_cache", ctypes.c_void_p), ("kv_dtype", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("scale_mode", ctypes.c_int32),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("sinks", ctypes.c_void_p), ("softmax_scale", ctypes.c_float),
                ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


class msa_index_cache(ctypes.Structure):
    _fields_ = [("k_cache", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("dtype", ctypes.c_int32), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32)]


class msa_mla_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("num_rows", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("dqk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("kv_cache", ctypes.c_void_p), ("num_tokens", ctypes.c_int64),
                ("kv_indptr", ctypes.c_void_p), ("kv_indices", ctypes.c_void_p),
                ("max_tokens", ctypes.c_int32), ("sinks", ctypes.c_void_p),
                ("softmax_scale", ctypes.c_float), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("q_dtype", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("q_scale", ctypes.c_void_p),
                ("kv_scale", ctypes.c_void_p)]


class msa_tree(ctypes.Structure):
    _fields_ = [("mask", ctypes.c_void_p), ("mask_words", ctypes.c_int32),
                ("topk_idx", ctypes.c_void_p), ("topk", ctypes.c_int32)]


class msa_cache_view(ctypes.Structure):
    _fields_ = [("lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("bt_stride", ctypes.c_int32), ("num_reqs", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("blocks", ctypes.c_void_p),
                ("refs", ctypes.c_void_p)]


class msa_kv_pools(ctypes.Structure):
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("kv_dtype", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("scale_mode", ctypes.c_int32),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("index", ctypes.c_void_p), ("mass", ctypes.c_void_p)]


class msa_rope(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("max_pos", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("positions", ctypes.c_void_p)]


class msa_qkv(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("idx_q", ctypes.c_void_p), ("idx_k", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("idx_q_stride", ctypes.c_int64),
                ("idx_k_stride", ctypes.c_int64), ("num_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
                ("idx_q_norm", ctypes.c_void_p), ("idx_k_norm", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("norm_shift", ctypes.c_float),
                ("q_out", ctypes.c_void_p), ("idx_q_out", ctypes.c_void_p)]


class msa_page_set(ctypes.Structure):
    _fields_ = [("lens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("refs", ctypes.c_void_p), ("copy_src", ctypes.c_void_p),
                ("copy_dst", ctypes.c_void_p), ("copy_tokens", ctypes.c_void_p),
                ("bt_stride", ctypes.c_int32), ("num_reqs", ctypes.c_int32),
                ("blocks", ctypes.c_void_p)]


class msa_trace(ctypes.Structure):
    _fields_ = [("after_score", ctypes.c_void_p), ("after_topk", ctypes.c_void_p),
                ("after_attn", ctypes.c_void_p), ("kernels", ctypes.c_int32)]


_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None


def library_path() -> str:
    return _build.LIB


def lib(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libmsa.so (building it first if asked and needed)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if build_if_missing and not _build.up_to_date():
                _build.build()
            if not os.path.exists(path):
                raise RuntimeError(f"libmsa.so not built ({path}); run "
                                   "python -m block_sparse_paged_02_gb300.build")
            L = ctypes.CDLL(path)
            P, i32 = ctypes.c_void_p, ctypes.c_int32
            L.msa_index_score.restype = ctypes.c_int
            L.msa_index_score.argtypes = [P, P, P, P, i32, P, P]
            L.msa_topk_build_table.restype = ctypes.c_int
            L.msa_topk_build_table.argtypes = [P, P, i32, i32, P, P, i32, P, P, P]
            L.msa_sparse_paged_attn.restype = ctypes.c_int
            L.msa_sparse_paged_attn.argtypes = [P, P, i32, P, P, ctypes.c_size_t, P, P]
            L.msa_decode.restype = ctypes.c_int
            L.msa_decode.argtypes = [P, P, P, i32, P, P, P, i32, P, P, ctypes.c_size_t, P, P, P]
            L.msa_kv_insert.restype = ctypes.c_int
            L.msa_kv_insert.argtypes = [P, P, P, i32, i32, P, P, i32, i32, P, P, P, P, i32, P,
                                        P]
            L.msa_sparse_mla_workspace_size.restype = ctypes.c_size_t
            L.msa_sparse_mla_workspace_size.argtypes = [i32, i32, i32]
            L.msa_sparse_mla_decode.restype = ctypes.c_int
            L.msa_sparse_mla_decode.argtypes = [P, P, ctypes.c_size_t, P, P]
            L.msa_workspace_size.restype = ctypes.c_size_t
            L.msa_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
            L.msa_check_bounded_wait.restype = ctypes.c_int
            L.msa_check_bounded_wait.argtypes = [P, ctypes.c_uint32, i32, P, P]
            L.msa_tree_attn_workspace_size.restype = ctypes.c_size_t
            L.msa_tree_attn_workspace_size.argtypes = [i32] * 6
            L.msa_tree_attn.restype = ctypes.c_int
            L.msa_tree_attn.argtypes = [P, P, P, P, ctypes.c_size_t, P, P]
            L.msa_attn_mass.restype = ctypes.c_int
            L.msa_attn_mass.argtypes = [P, P, P, P, P, ctypes.c_size_t, P, P]
            L.msa_evict_select.restype = ctypes.c_int
            L.msa_evict_select.argtypes = [P, P, i32, i32, i32, P, P, P, P]
            L.msa_kv_compact.restype = ctypes.c_int
            L.msa_kv_compact.argtypes = [P, P, P, i32, P, P, P, P]
            L.msa_qk_rope_insert.restype = ctypes.c_int
            L.msa_qk_rope_insert.argtypes = [P, P, P, P, P, P]
            L.msa_prompt_attn_workspace_size.restype = ctypes.c_size_t
            L.msa_prompt_attn_workspace_size.argtypes = [i32, i32]
            L.msa_prompt_attn.restype = ctypes.c_int
            L.msa_prompt_attn.argtypes = [P, P, P, ctypes.c_size_t, P, P]
            L.msa_page_fork.restype = ctypes.c_int
            L.msa_page_fork.argtypes = [P, P, P, P, P, P, P]
            L.msa_page_copy.restype = ctypes.c_int
            L.msa_page_copy.argtypes = [P, i32, i32, P, P, P, i32, P, P]
            L.msa_status_string.restype = ctypes.c_char_p
            L.msa_status_string.argtypes = [ctypes.c_int]
            _lib = L
    return _lib


def msa_status_string(code: int) -> str:
    return lib().msa_status_string(int(code)).decode()


status_string = msa_status_string


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libmsa takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libmsa takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _one_device(*tensors: Optional[torch.Tensor]):
    """The tensors of one argument structure live on one device."""
    there = {t.device for t in tensors if t is not None}
    if len(there) > 1:
        raise ValueError(f"tensors on different devices: {', '.join(sorted(map(str, there)))}")


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(fn: str, code: int):
    if code != MSA_OK:
        raise MsaError(fn, code)


def make_batch(cu_seqlens_q, cu_seqlens_k, context_lens, block_table, num_pages: int,
               num_rows: Optional[int] = None, max_q_len: int = 0,
               min_q_len: int = 0) -> msa_batch:
    for t in (cu_seqlens_q, cu_seqlens_k, context_lens, block_table):
        if t.dtype != torch.int32:
            raise ValueError("batch geometry arrays are int32")
    _one_device(cu_seqlens_q, cu_seqlens_k, context_lens, block_table)
    b = msa_batch(_p(cu_seqlens_q), _p(cu_seqlens_k), _p(context_lens), _p(block_table),
                  int(block_table.shape[1]), int(context_lens.shape[0]),
                  int(num_rows if num_rows is not None else 0), int(num_pages), int(max_q_len),
                  int(min_q_len))
    b._keep = (cu_seqlens_q, cu_seqlens_k, context_lens, block_table)
    return b


def check_sinks(sinks: Optional[torch.Tensor], num_heads: int):
    """Sink contract of the sparse-MLA sink PR: fp32, 1-D, num_heads long,
    contiguous -- a C ABI cannot see dtypes, so it is checked here."""
    if sinks is None:
        return
    if sinks.dtype != torch.float32:
        raise ValueError(f"sinks must be float32, got {sinks.dtype}")
    if sinks.ndim != 1 or sinks.numel() != num_heads:
        raise ValueError(f"sinks must have shape ({num_heads},), got {tuple(sinks.shape)}")
    if not sinks.is_contiguous():
        raise ValueError("sinks must be contiguous")


def make_index_cache(k_cache, dtype: int = MSA_KV_BF16, k_scale=None) -> msa_index_cache:
    """The paged index-K cache [P, 128, heads, dim] (bf16, or e4m3 codes with
    optional fp32 per-token scales [P, 128, heads])."""
    _one_device(k_cache, k_scale)
    x = msa_index_cache(_p(k_cache), _p(k_scale), int(dtype), int(k_cache.shape[2]),
                        int(k_cache.shape[3]))
    x._keep = (k_cache, k_scale)
    return x


def make_attn_args(q, k_cache, v_cache, kv_dtype: int, num_pages: int, out, lse, *,
                   scale_mode: int = MSA_SCALE_NONE, k_scale=None, v_scale=None, sinks=None,
                   softmax_scale: float) -> msa_attn_args:
    check_sinks(sinks, int(q.shape[1]))
    _one_device(q, k_cache, v_cache, out, lse, k_scale, v_scale, sinks)
    a = msa_attn_args(_p(q), int(q.shape[0]), int(q.shape[1]), int(k_cache.shape[-2]),
                      int(q.shape[2]), _p(k_cache), _p(v_cache), int(kv_dtype), int(num_pages),
                      int(scale_mode), _p(k_scale), _p(v_scale), _p(sinks),
                      float(softmax_scale), _p(out), _p(lse))
    a._keep = (q, k_cache, v_cache, out, lse, k_scale, v_scale, sinks)
    return a


# ------------------------------------------------------------- entry points

def msa_workspace_size(num_rows, bt_stride, topk, num_heads, head_dim, tbl_stride) -> int:
    return int(lib().msa_workspace_size(int(num_rows), int(bt_stride), int(topk),
                                        int(num_heads), int(head_dim), int(tbl_stride)))


def msa_index_score(batch: msa_batch, idx_q, index: msa_index_cache, scores, score_stride,
                    dev_status, stream=None):
    _check("msa_index_score", lib().msa_index_score(
        ctypes.byref(batch), _p(idx_q), ctypes.byref(index), _p(scores), int(score_stride),
        _p(dev_status), _stream(stream)))


def msa_topk_build_table(batch: msa_batch, scores, score_stride, topk, topk_idx, sparse_tbl,
                         tbl_stride, sparse_len, dev_status, stream=None):
    _check("msa_topk_build_table", lib().msa_topk_build_table(
        ctypes.byref(batch), _p(scores), int(score_stride), int(topk), _p(topk_idx),
        _p(sparse_tbl), int(tbl_stride), _p(sparse_len), _p(dev_status), _stream(stream)))


def msa_sparse_paged_attn(attn: msa_attn_args, sparse_tbl, tbl_stride, sparse_len, workspace,
                          dev_status, stream=None):
    _check("msa_sparse_paged_attn", lib().msa_sparse_paged_attn(
        ctypes.byref(attn), _p(sparse_tbl), int(tbl_stride), _p(sparse_len), _p(workspace),
        int(workspace.numel() * workspace.element_size()) if workspace is not None else 0,
        _p(dev_status), _stream(stream)))


def msa_decode(batch: msa_batch, idx_q, index: msa_index_cache, topk, attn: msa_attn_args,
               topk_idx, sparse_tbl, tbl_stride, sparse_len, workspace, dev_status,
               trace: Optional[msa_trace] = None, stream=None):
    _check("msa_decode", lib().msa_decode(
        ctypes.byref(batch), _p(idx_q), ctypes.byref(index), int(topk), ctypes.byref(attn),
        _p(topk_idx), _p(sparse_tbl), int(tbl_stride), _p(sparse_len), _p(workspace),
        int(workspace.numel() * workspace.element_size()) if workspace is not None else 0,
        _p(dev_status), ctypes.byref(trace) if trace is not None else None, _stream(stream)))


def msa_kv_insert(batch: msa_batch, k_new, v_new, num_kv_heads, head_dim, k_cache, v_cache,
                  kv_dtype, scale_mode, k_scale, v_scale, idx_new,
                  index: Optional[msa_index_cache], skip_index, dev_status, stream=None):
    _check("msa_kv_insert", lib().msa_kv_insert(
        ctypes.byref(batch), _p(k_new), _p(v_new), int(num_kv_heads), int(head_dim),
        _p(k_cache), _p(v_cache), int(kv_dtype), int(scale_mode), _p(k_scale), _p(v_scale),
        _p(idx_new), ctypes.byref(index) if index is not None else None,
        int(bool(skip_index)), _p(dev_status), _stream(stream)))


def make_mla_args(q, kv_cache, kv_indptr, kv_indices, out, lse, *, max_tokens: int,
                  sinks=None, softmax_scale: float, q_scale=None,
                  kv_scale=None) -> msa_mla_args:
    """Sparse MLA operands: q [N, H, 576] bf16 (or uint8 e4m3 codes with
    q_scale), kv_cache [T, 576] bf16 (or uint8 e4m3 codes with kv_scale),
    int32 kv_indptr [N+1] / kv_indices, out [N, H, 512] bf16, lse [N, H]
    fp32; scales are device fp32 [1]."""
    check_sinks(sinks, int(q.shape[1]))
    for t in (kv_indptr, kv_indices):
        if t.dtype != torch.int32:
            raise ValueError("kv_indptr / kv_indices are int32")
    q8 = q.dtype == torch.uint8
    kv8 = kv_cache.dtype == torch.uint8
    a = msa_mla_args(_p(q), int(q.shape[0]), int(q.shape[1]), int(q.shape[2]),
                     int(out.shape[2]), _p(kv_cache), int(kv_cache.shape[0]), _p(kv_indptr),
                     _p(kv_indices), int(max_tokens), _p(sinks), float(softmax_scale), _p(out),
                     _p(lse), MSA_KV_FP8_E4M3 if q8 else MSA_KV_BF16,
                     MSA_KV_FP8_E4M3 if kv8 else MSA_KV_BF16, _p(q_scale), _p(kv_scale))
    a._keep = (q, kv_cache, kv_indptr, kv_indices, out, lse, sinks, q_scale, kv_scale)
    return a


def msa_sparse_mla_workspace_size(num_rows, num_heads, max_tokens) -> int:
    return int(lib().msa_sparse_mla_workspace_size(int(num_rows), int(num_heads),
                                                   int(max_tokens)))


def msa_sparse_mla_decode(mla: msa_mla_args, workspace, dev_status, stream=None):
    _check("msa_sparse_mla_decode", lib().msa_sparse_mla_decode(
        ctypes.byref(mla), _p(workspace),
        int(workspace.numel() * workspace.element_size()) if workspace is not None else 0,
        _p(dev_status), _stream(stream)))


def msa_check_bounded_wait(dev_status, limit_us: int, flags: int = 0, copy_src=None,
                           stream=None):
    """Run the bounded-wait check (see msa.h): a wait that nothing satisfies
    gives up after limit_us and sets MSA_DEV_TIMEOUT in dev_status."""
    _check("msa_check_bounded_wait", lib().msa_check_bounded_wait(
        _p(dev_status), int(limit_us), int(flags), _p(copy_src), _stream(stream)))


# ------------------------------------ draft trees and eviction (msa_cache.h)

def _typed(name: str, t: Optional[torch.Tensor], dtypes, shape=None):
    """The tensor's type and shape (None: any extent), which a C ABI cannot see."""
    if t is None:
        return
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if shape is not None and t.shape != shape and (
            t.ndim != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape))):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


# The calls of this part are made once per layer and step: pointers go through
# ctypes as plain integers, and the stream is the current one's raw handle.

def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libmsa takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libmsa takes contiguous tensors")
    return t.data_ptr()


def _on(stream, *tensors: Optional[torch.Tensor]) -> int:
    """The raw stream of a call on the current device, on which its tensors have to live."""
    device = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"tensor on {t.device}, but cuda:{device} is current")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _first(struct) -> Optional[torch.Tensor]:
    """A tensor behind an argument structure that this module made (all are on its device)."""
    for t in getattr(struct, "_keep", ()):
        if t is not None:
            return t
    return None


def _calls() -> ctypes.CDLL:
    return _lib if _lib is not None else lib()


def make_tree(mask: Optional[torch.Tensor] = None,
              topk_idx: Optional[torch.Tensor] = None) -> msa_tree:
    """What the drafted rows see: `mask` int32 or uint32 [num_rows, words] (bit i of a row: it
    sees drafted token i; None: a causal chain) and `topk_idx` int32 [num_rows, topk] (the
    row's selected blocks; None: the whole context)."""
    _typed("mask", mask, (torch.int32, torch.uint32), (None, None))
    _typed("topk_idx", topk_idx, (torch.int32,), (None, None))
    _one_device(mask, topk_idx)
    t = msa_tree(_p(mask), int(mask.shape[1]) if mask is not None else 0, _p(topk_idx),
                 int(topk_idx.shape[1]) if topk_idx is not None else 0)
    t._keep = (mask, topk_idx)
    return t


def _tree_rows(batch: msa_batch, tree: msa_tree):
    mask, topk_idx = tree._keep
    if mask is not None and mask.shape[0] != batch.num_rows:
        raise ValueError(f"mask has {mask.shape[0]} rows, the batch {batch.num_rows}")
    if topk_idx is not None and topk_idx.shape[0] != batch.num_rows:
        raise ValueError(f"topk_idx has {topk_idx.shape[0]} rows, the batch {batch.num_rows}")


def msa_tree_attn_workspace_size(num_reqs, num_rows, bt_stride, num_heads, max_q_len=0,
                                 topk=0) -> int:
    return int(lib().msa_tree_attn_workspace_size(int(num_reqs), int(num_rows), int(bt_stride),
                                                  int(num_heads), int(max_q_len), int(topk)))


def _bytes(t: Optional[torch.Tensor]) -> int:
    return t.nbytes if t is not None else 0


def msa_tree_attn(batch: msa_batch, tree: msa_tree, attn: msa_attn_args, workspace, dev_status,
                  stream=None):
    """Attention of every drafted row over its request's cache (see msa_cache.h)."""
    _tree_rows(batch, tree)
    ws, st = _ptr(workspace), _ptr(dev_status)
    _check("msa_tree_attn", _calls().msa_tree_attn(
        ctypes.byref(batch), ctypes.byref(tree), ctypes.byref(attn), ws, _bytes(workspace), st,
        _on(stream, dev_status, workspace, _first(batch), _first(tree), _first(attn))))


def msa_attn_mass(batch: msa_batch, tree: msa_tree, attn: msa_attn_args, mass, workspace,
                  dev_status, stream=None):
    """Add the weight that each cached token received to `mass` fp32 [num_pages, 128]; the rows'
    log-sum-exps are read from the attention arguments' lse."""
    _tree_rows(batch, tree)
    _typed("mass", mass, (torch.float32,), (batch.num_pages, 128))
    m, ws, st = _ptr(mass), _ptr(workspace), _ptr(dev_status)
    _check("msa_attn_mass", _calls().msa_attn_mass(
        ctypes.byref(batch), ctypes.byref(tree), ctypes.byref(attn), m, ws, _bytes(workspace), st,
        _on(stream, dev_status, workspace, mass, _first(batch), _first(tree), _first(attn))))


def make_cache_view(lens, block_table, num_pages: int, blocks=None, refs=None) -> msa_cache_view:
    """The cached tokens of a set of requests: int32 lens [R], block_table [R, bt_stride]; for
    msa_page_fork blocks [R], the pages that each holds (None: those of its tokens); for
    msa_kv_compact refs [num_pages], by which requests that share pages are refused."""
    _typed("lens", lens, (torch.int32,), (None,))
    _typed("block_table", block_table, (torch.int32,), (int(lens.shape[0]), None))
    _typed("blocks", blocks, (torch.int32,), (int(lens.shape[0]),))
    _typed("refs", refs, (torch.int32,), (int(num_pages),))
    _one_device(lens, block_table, blocks, refs)
    c = msa_cache_view(_p(lens), _p(block_table), int(block_table.shape[1]), int(lens.shape[0]),
                       int(num_pages), _p(blocks), _p(refs))
    c._keep = (lens, block_table, blocks, refs)
    return c


def msa_evict_select(cache: msa_cache_view, mass, budget: int, keep_first: int, keep_recent: int,
                     keep, keep_len, dev_status, stream=None):
    """The positions each request keeps under the budget, into keep int32 [R, budget] (ascending,
    then -1) and keep_len int32 [R]."""
    _typed("mass", mass, (torch.float32,), (cache.num_pages, 128))
    _typed("keep", keep, (torch.int32,), (cache.num_reqs, int(budget)))
    _typed("keep_len", keep_len, (torch.int32,), (cache.num_reqs,))
    m, k, n, st = _ptr(mass), _ptr(keep), _ptr(keep_len), _ptr(dev_status)
    _check("msa_evict_select", _calls().msa_evict_select(
        ctypes.byref(cache), m, int(budget), int(keep_first), int(keep_recent), k, n, st,
        _on(stream, dev_status, mass, keep, keep_len, _first(cache))))


def make_kv_pools(k_cache, v_cache, kv_dtype: int, *, scale_mode: int = MSA_SCALE_NONE,
                  k_scale=None, v_scale=None, index: Optional[msa_index_cache] = None,
                  mass=None) -> msa_kv_pools:
    """The pools whose tokens move together: K and V [P, 128, Hkv, 128], per-token-head scales
    [P, 128, Hkv], an index cache of make_index_cache, accumulated weights [P, 128]."""
    pages, _, hkv, dim = (int(x) for x in k_cache.shape)
    of = (torch.uint8, torch.float8_e4m3fn) if kv_dtype == MSA_KV_FP8_E4M3 else (torch.bfloat16,)
    _typed("k_cache", k_cache, of, (pages, 128, hkv, dim))
    _typed("v_cache", v_cache, of, (pages, 128, hkv, dim))
    if scale_mode == MSA_SCALE_PER_TOKEN_HEAD:
        _typed("k_scale", k_scale, (torch.float32,), (pages, 128, hkv))
        _typed("v_scale", v_scale, (torch.float32,), (pages, 128, hkv))
    _typed("mass", mass, (torch.float32,), (pages, 128))
    if index is not None:
        ik, iscale = index._keep
        if int(ik.shape[0]) != pages:
            raise ValueError(f"the index cache has {ik.shape[0]} pages, K has {pages}")
        of = (torch.uint8, torch.float8_e4m3fn) if index.dtype == MSA_KV_FP8_E4M3 else (torch.bfloat16,)
        _typed("index k_cache", ik, of, (pages, 128, index.heads, index.dim))
        _typed("index k_scale", iscale, (torch.float32,), (pages, 128, index.heads))
    _one_device(k_cache, v_cache, k_scale, v_scale, mass, *(index._keep if index is not None else ()))
    x = msa_kv_pools(_p(k_cache), _p(v_cache), int(kv_dtype), hkv, dim, int(scale_mode),
                     _p(k_scale), _p(v_scale),
                     ctypes.cast(ctypes.pointer(index), ctypes.c_void_p) if index is not None else None,
                     _p(mass))
    x._keep = (k_cache, v_cache, k_scale, v_scale, index, mass)
    x._pages = pages
    return x


def msa_kv_compact(cache: msa_cache_view, base, keep, keep_len, pools: msa_kv_pools, dev_status,
                   stream=None):
    """Move the tokens at base + keep[r, i] to base + i, i < keep_len[r], in every pool (base
    int32 [R] or None for 0; keep int32 [R, stride], strictly ascending; keep_len int32 [R])."""
    _typed("base", base, (torch.int32,), (cache.num_reqs,))
    _typed("keep", keep, (torch.int32,), (cache.num_reqs, None))
    _typed("keep_len", keep_len, (torch.int32,), (cache.num_reqs,))
    if pools._pages != cache.num_pages:
        raise ValueError(f"the pools have {pools._pages} pages, the cache view {cache.num_pages}")
    b, k, n, st = _ptr(base), _ptr(keep), _ptr(keep_len), _ptr(dev_status)
    _check("msa_kv_compact", _calls().msa_kv_compact(
        ctypes.byref(cache), b, k, keep.shape[1], n, ctypes.byref(pools), st,
        _on(stream, dev_status, base, keep, keep_len, _first(cache), _first(pools))))


# -------------------------------- prompts and shared pages (msa_prompt.h)

def _rows_of(name: str, t: Optional[torch.Tensor], heads=None, dim=None):
    """Pointer, row stride and shape of bf16 vectors [N, heads, dim] whose rows may lie apart (a
    slice of a projection's output); a row's heads are packed."""
    if t is None:
        return None, 0
    _typed(name, t, (torch.bfloat16,), (None, heads, dim))
    if not t.is_cuda:
        raise ValueError("libmsa takes device tensors")
    n, h, d = t.shape
    if (d > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != d):
        raise ValueError(f"{name}: the heads of a row must be packed, got strides {t.stride()}")
    return t.data_ptr(), t.stride(0) if n > 1 else h * d


def make_rope(cos_sin: Optional[torch.Tensor], *, interleaved: bool = False,
              positions: Optional[torch.Tensor] = None) -> msa_rope:
    """The rotation: cos_sin fp32 [max_pos, rotary_dim] (cosines, then sines; None: none),
    `interleaved` pairs neighbours instead of halves, positions int32 [num_rows] (None: the
    rows' places in the cache)."""
    _typed("cos_sin", cos_sin, (torch.float32,), (None, None))
    _typed("positions", positions, (torch.int32,), (None,))
    _one_device(cos_sin, positions)
    r = msa_rope(_p(cos_sin), int(cos_sin.shape[0]) if cos_sin is not None else 0,
                 int(cos_sin.shape[1]) if cos_sin is not None else 0, int(bool(interleaved)),
                 _p(positions))
    r._keep = (cos_sin, positions)
    return r


def make_qkv(q, k, v, q_out, *, idx_q=None, idx_k=None, idx_q_out=None, q_norm=None, k_norm=None,
             idx_q_norm=None, idx_k_norm=None, eps: float = 1e-6, norm_shift: float = 0.0) -> msa_qkv:
    """The new tokens' vectors: q [N, H, 128], k and v [N, Hkv, 128], idx_q and idx_k [N, Hi, Di]
    bf16 (rows may lie apart), their RMS-norm weights bf16 [dim] (None: not normed), and the
    packed outputs q_out, idx_q_out bf16 (q_out may be a packed q itself)."""
    n, h, d = (int(x) for x in q.shape)
    hk = int(k.shape[1])
    if k.shape[0] != n:
        raise ValueError(f"k has {k.shape[0]} rows, q {n}")
    qp, qs = _rows_of("q", q)
    kp, ks = _rows_of("k", k, None, d)
    vp, vs = _rows_of("v", v, hk, d)
    _typed("q_out", q_out, (torch.bfloat16,), (n, h, d))
    _typed("v", v, (torch.bfloat16,), (n, hk, d))
    ip = jp = None
    istr = jstr = 0
    if (idx_q is None) != (idx_k is None) or (idx_q is None) != (idx_q_out is None):
        raise ValueError("idx_q, idx_k and idx_q_out come together")
    if idx_q is not None:
        hi, di = int(idx_q.shape[1]), int(idx_q.shape[2])
        _typed("idx_q", idx_q, (torch.bfloat16,), (n, hi, di))
        _typed("idx_k", idx_k, (torch.bfloat16,), (n, hi, di))
        _typed("idx_q_out", idx_q_out, (torch.bfloat16,), (n, hi, di))
        ip, istr = _rows_of("idx_q", idx_q)
        jp, jstr = _rows_of("idx_k", idx_k)
        for name, w in (("idx_q_norm", idx_q_norm), ("idx_k_norm", idx_k_norm)):
            _typed(name, w, (torch.bfloat16,), (di,))
    for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
        _typed(name, w, (torch.bfloat16,), (d,))
    for src, stride, out in ((q, qs, q_out), (idx_q, istr, idx_q_out)):
        if src is not None and n > 1 and out.data_ptr() == src.data_ptr() and stride != src.shape[1] * src.shape[2]:
            raise ValueError("an output in place of its input needs packed rows")
    _one_device(q, k, v, q_out, idx_q, idx_k, idx_q_out, q_norm, k_norm, idx_q_norm, idx_k_norm)
    x = msa_qkv(qp, kp, vp, ip, jp, qs, ks, vs, istr, jstr, h, hk, d, _p(q_norm), _p(k_norm),
                _p(idx_q_norm), _p(idx_k_norm), float(eps), float(norm_shift), _p(q_out), _p(idx_q_out))
    x._keep = (q, k, v, q_out, idx_q, idx_k, idx_q_out, q_norm, k_norm, idx_q_norm, idx_k_norm)
    x._rows = n
    x._index = None if idx_q is None else tuple(idx_q.shape[1:])
    return x


def msa_qk_rope_insert(batch: msa_batch, qkv: msa_qkv, rope: msa_rope, pools: msa_kv_pools, dev_status,
                       stream=None):
    """Norm, rotation and insertion of the rows' vectors in one pass (see msa_prompt.h); `pools`
    as make_kv_pools makes them (an e4m3 pool with one scale takes fp32 [1] k_scale and v_scale)."""
    if qkv._rows != batch.num_rows:
        raise ValueError(f"the vectors have {qkv._rows} rows, the batch {batch.num_rows}")
    positions = rope._keep[1]
    if positions is not None and positions.shape[0] != batch.num_rows:
        raise ValueError(f"positions has {positions.shape[0]} rows, the batch {batch.num_rows}")
    if pools._pages != batch.num_pages:
        raise ValueError(f"the pools have {pools._pages} pages, the batch {batch.num_pages}")
    k_scale, v_scale, index = pools._keep[2:5]
    if pools.scale_mode == MSA_SCALE_SCALAR:
        _typed("k_scale", k_scale, (torch.float32,), (1,))
        _typed("v_scale", v_scale, (torch.float32,), (1,))
    if index is not None and qkv._index != (index.heads, index.dim):
        raise ValueError(f"index vectors {qkv._index}, index cache {(index.heads, index.dim)}")
    st = _ptr(dev_status)
    _check("msa_qk_rope_insert", _calls().msa_qk_rope_insert(
        ctypes.byref(batch), ctypes.byref(qkv), ctypes.byref(rope), ctypes.byref(pools), st,
        _on(stream, dev_status, _first(batch), _first(qkv), _first(rope), _first(pools))))


def msa_prompt_attn_workspace_size(num_heads, num_kv_heads) -> int:
    return int(lib().msa_prompt_attn_workspace_size(int(num_heads), int(num_kv_heads)))


def msa_prompt_attn(batch: msa_batch, attn: msa_attn_args, workspace, dev_status, stream=None):
    """Causal attention of whole prompts or their chunks over the cache (see msa_prompt.h)."""
    ws, st = _ptr(workspace), _ptr(dev_status)
    _check("msa_prompt_attn", _calls().msa_prompt_attn(
        ctypes.byref(batch), ctypes.byref(attn), ws, _bytes(workspace), st,
        _on(stream, dev_status, workspace, _first(batch), _first(attn))))


def make_page_set(lens, block_table, refs, copy_src, copy_dst, copy_tokens, blocks=None) -> msa_page_set:
    """What msa_page_fork writes: int32 lens [R], block_table [R, bt_stride], refs [num_pages], the
    pages to copy, copy_src, copy_dst, copy_tokens [R], and (where given) the pages held, blocks [R]."""
    n = int(lens.shape[0])
    _typed("lens", lens, (torch.int32,), (None,))
    _typed("block_table", block_table, (torch.int32,), (n, None))
    _typed("refs", refs, (torch.int32,), (None,))
    for name, t in (("copy_src", copy_src), ("copy_dst", copy_dst), ("copy_tokens", copy_tokens),
                    ("blocks", blocks)):
        _typed(name, t, (torch.int32,), (n,))
    every = (lens, block_table, refs, copy_src, copy_dst, copy_tokens)
    _one_device(*every, blocks)
    x = msa_page_set(*(_p(t) for t in every), int(block_table.shape[1]), n, _p(blocks))
    x._keep = every
    x._blocks = blocks
    return x


def msa_page_fork(cache: msa_cache_view, refs, parent, grow, to: msa_page_set, dev_status, stream=None):
    """The requests that go on and their pages: request i of `to` continues request parent[i] of
    `cache` (-1: a new one) and is about to write grow[i] tokens (see msa_prompt.h)."""
    _typed("refs", refs, (torch.int32,), (cache.num_pages,))
    _typed("parent", parent, (torch.int32,), (to.num_reqs,))
    _typed("grow", grow, (torch.int32,), (to.num_reqs,))
    if to._keep[2].shape[0] != cache.num_pages:
        raise ValueError(f"the set counts {to._keep[2].shape[0]} pages, the cache view {cache.num_pages}")
    r, p, g, st = _ptr(refs), _ptr(parent), _ptr(grow), _ptr(dev_status)
    _check("msa_page_fork", _calls().msa_page_fork(
        ctypes.byref(cache), r, p, g, ctypes.byref(to), st,
        _on(stream, dev_status, refs, parent, grow, _first(cache), _first(to))))


def msa_page_copy(layers, src, dst, tokens, dev_status, stream=None):
    """Copy the first tokens[i] slots of page src[i] to page dst[i] (int32 [n]) in the pools of
    every layer (a sequence of make_kv_pools structs of as many pages each)."""
    layers = list(layers)
    pages = {x._pages for x in layers}
    if len(pages) > 1:
        raise ValueError(f"layers of different numbers of pages: {sorted(pages)}")
    _typed("src", src, (torch.int32,), (None,))
    n = src.shape[0]
    _typed("dst", dst, (torch.int32,), (n,))
    _typed("tokens", tokens, (torch.int32,), (n,))
    s, d, t, st = _ptr(src), _ptr(dst), _ptr(tokens), _ptr(dev_status)
    _check("msa_page_copy", _calls().msa_page_copy(
        b"".join(layers), len(layers), pages.pop() if pages else 0, s, d, t, n, st,
        _on(stream, dev_status, src, dst, tokens, *(_first(x) for x in layers))))


def make_trace(after_score=None, after_topk=None, after_attn=None) -> msa_trace:
    """Events (torch.cuda.Event, created with enable_timing) that msa_decode
    records after each stage.  torch creates an event lazily on its first
    record, so each is recorded once here to obtain its handle."""
    for e in (after_score, after_topk, after_attn):
        if e is not None and not e.cuda_event:
            e.record()
    h = lambda e: ctypes.c_void_p(e.cuda_event) if e is not None else None
    t = msa_trace(h(after_score), h(after_topk), h(after_attn), 0)
    t._keep = (after_score, after_topk, after_attn)
    return t
