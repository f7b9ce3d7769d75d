"""ctypes binding of libvt (include/vt.h).  Argument marshalling only.

Every function takes CUDA torch tensors, passes their device pointers, sizes and strides to
the C entry point of the same name, and enqueues on the current torch CUDA stream.  All
computation happens in libvt's kernels; there is no fallback of any kind: if libvt.so is
missing or a call fails, a ``VtError`` is raised.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libvt.so")

VT_OK, VT_ERR_INVALID_ARG, VT_ERR_UNSUPPORTED, VT_ERR_CUDA = 0, 1, 2, 3
VT_DEV_BAD_PAGE, VT_DEV_BAD_LEN, VT_DEV_BAD_SEL, VT_DEV_BAD_ORDER, VT_DEV_TIMEOUT = 1, 2, 4, 8, 16
VT_DEV_BAD_START, VT_DEV_NO_PAGE, VT_DEV_BAD_REF, VT_DEV_BAD_REQ = 32, 64, 128, 256
PAGE_SIZE = 16


class VtError(RuntimeError):
    def __init__(self, code: int, where: str, detail: str):
        super().__init__(f"{where}: {_status_name(code)}: {detail}")
        self.code = code


class PagedKV(ctypes.Structure):
    _fields_ = [
        ("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
        ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("head_dim_v", ctypes.c_int32),
        ("sk_p", ctypes.c_int64), ("sk_t", ctypes.c_int64), ("sk_h", ctypes.c_int64),
        ("sv_p", ctypes.c_int64), ("sv_t", ctypes.c_int64), ("sv_h", ctypes.c_int64),
    ]


class DecodeArgs(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("pt_stride", ctypes.c_int64),
        ("seq_lens", ctypes.c_void_p), ("centroids", ctypes.c_void_p),
        ("topk", ctypes.c_int32), ("bos", ctypes.c_int32), ("eos", ctypes.c_int32),
        ("sm_scale", ctypes.c_float),
        ("order", ctypes.c_void_p), ("status", ctypes.c_void_p),
    ]


class PrefillArgs(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
        ("num_tokens", ctypes.c_int64), ("q", ctypes.c_void_p), ("sq_t", ctypes.c_int64),
        ("q_start", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
        ("pt_stride", ctypes.c_int64), ("seq_lens", ctypes.c_void_p),
        ("sm_scale", ctypes.c_float), ("status", ctypes.c_void_p), ("max_pages", ctypes.c_int64),
    ]


class SharedPrefixArgs(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
        ("num_groups", ctypes.c_int32), ("q", ctypes.c_void_p),
        ("group_start", ctypes.c_void_p), ("prefix_pages", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p), ("pt_stride", ctypes.c_int64),
        ("seq_lens", ctypes.c_void_p), ("sm_scale", ctypes.c_float),
        ("status", ctypes.c_void_p), ("max_pages", ctypes.c_int64),
    ]


class PageBooks(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int32), ("page_table", ctypes.c_void_p), ("pt_stride", ctypes.c_int64),
        ("seq_lens", ctypes.c_void_p), ("refs", ctypes.c_void_p), ("status", ctypes.c_void_p),
        ("max_pages", ctypes.c_int64),
    ]


EXPORTS = ("vt_build_centroids", "vt_select_pages", "vt_select_pages_approx",
           "vt_select_pages_ws", "vt_sparse_decode_ws",
           "vt_sparse_decode", "vt_sparse_decode_fused", "vt_sparse_decode_step",
           "vt_fused_workspace_size", "vt_sparse_decode_fused_static", "vt_plan_requests",
           "vt_prefill", "vt_prefill_workspace_size", "vt_shared_prefix_decode",
           "vt_shared_prefix_workspace_size", "vt_copy_pages", "vt_fork_requests",
           "vt_extend_requests", "vt_free_requests", "vt_compact_pages",
           "vt_page_workspace_size",
           "vt_status_string",
           "vt_last_error_detail", "vt_abi_version")

_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH):
    """Load libvt.so (once).  Raises VtError if it is missing: there is no fallback."""
    global _lib
    lib = _lib
    if lib is not None:
        return lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise VtError(-1, "load", f"{path} not found; build it with "
                                          "`python -m paged_block_sparse_vt_b200.build`")
            lib = ctypes.CDLL(path)
            P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
            kv, args = ctypes.POINTER(PagedKV), ctypes.POINTER(DecodeArgs)
            prefill, shared = ctypes.POINTER(PrefillArgs), ctypes.POINTER(SharedPrefixArgs)
            books = ctypes.POINTER(PageBooks)
            sigs = {
                "vt_build_centroids": [kv, P, I32, P, P, P],
                "vt_select_pages": [kv, args, P, P, P],
                "vt_select_pages_approx": [kv, args, ctypes.c_uint64, P, P, P],
                "vt_select_pages_ws": [kv, args, P, P, P, ctypes.c_size_t, P],
                "vt_sparse_decode_ws": [kv, args, P, P, P, P, P, ctypes.c_size_t, P],
                "vt_sparse_decode": [kv, args, P, P, P, P, P],
                "vt_sparse_decode_fused": [kv, args, P, P, P, P, P, ctypes.c_size_t, P],
                "vt_sparse_decode_step": [kv, args, P, I32, P, P, P, P, P, P, ctypes.c_size_t, P],
                "vt_sparse_decode_fused_static": [kv, args, P, P, P, P, P],
                "vt_plan_requests": [P, I32, P, P],
                "vt_prefill": [kv, prefill, P, P, P, ctypes.c_size_t, P],
                "vt_shared_prefix_decode": [kv, shared, P, P, P, ctypes.c_size_t, P],
                "vt_copy_pages": [kv, P, P, I32, P, P, P],
                "vt_fork_requests": [kv, books, P, P, I32, P, ctypes.c_size_t, P],
                "vt_extend_requests": [books, I64, P, P, I32, P, ctypes.c_size_t, P],
                "vt_free_requests": [books, I64, P, I32, P],
                "vt_compact_pages": [kv, books, P, P, P, ctypes.c_size_t, P],
            }
            for name, argtypes in sigs.items():
                fn = getattr(lib, name)
                fn.argtypes = argtypes
                fn.restype = ctypes.c_int
            lib.vt_fused_workspace_size.argtypes = [kv, args]
            lib.vt_fused_workspace_size.restype = ctypes.c_size_t
            lib.vt_prefill_workspace_size.argtypes = [kv, prefill]
            lib.vt_prefill_workspace_size.restype = ctypes.c_size_t
            lib.vt_shared_prefix_workspace_size.argtypes = [kv, shared]
            lib.vt_shared_prefix_workspace_size.restype = ctypes.c_size_t
            lib.vt_page_workspace_size.argtypes = [I64, I32]
            lib.vt_page_workspace_size.restype = ctypes.c_size_t
            lib.vt_status_string.argtypes = [ctypes.c_int]
            lib.vt_status_string.restype = ctypes.c_char_p
            lib.vt_last_error_detail.argtypes = []
            lib.vt_last_error_detail.restype = ctypes.c_char_p
            lib.vt_abi_version.argtypes = []
            lib.vt_abi_version.restype = ctypes.c_int32
            _lib = lib
    return _lib


def _status_name(code: int) -> str:
    return {0: "VT_OK", 1: "VT_ERR_INVALID_ARG", 2: "VT_ERR_UNSUPPORTED", 3: "VT_ERR_CUDA"}.get(
        code, f"status {code}")


def _check(rc: int, where: str) -> None:
    if rc != VT_OK:
        detail = load_library().vt_last_error_detail().decode()
        raise VtError(rc, where, detail)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# The current stream's handle without building a torch.cuda.Stream object per call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t: torch.Tensor) -> int:
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _need(t: torch.Tensor, name: str, dtype=None, contiguous: bool = False) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise VtError(VT_ERR_INVALID_ARG, name, "must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise VtError(VT_ERR_INVALID_ARG, name, f"must be {dtype}, got {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise VtError(VT_ERR_INVALID_ARG, name, "must be contiguous")


def paged_kv(k_pool: torch.Tensor, v_pool: torch.Tensor, head_dim_v: Optional[int] = None) -> PagedKV:
    """Descriptor of the pools [P, 16, Hkv, D] (bf16, any strides with the last one 1)."""
    _need(k_pool, "k_pool", torch.bfloat16)
    _need(v_pool, "v_pool", torch.bfloat16)
    if k_pool.dim() != 4 or v_pool.dim() != 4:
        raise VtError(VT_ERR_INVALID_ARG, "pools", "must be [P, page_size, Hkv, D]")
    P, ps, hkv, d = k_pool.shape
    dv = head_dim_v if head_dim_v is not None else v_pool.shape[3]
    if k_pool.stride(3) != 1 or v_pool.stride(3) != 1:
        raise VtError(VT_ERR_UNSUPPORTED, "pools", "innermost stride must be 1")
    return PagedKV(k_pool.data_ptr(), v_pool.data_ptr(), P, ps, hkv, d, dv,
                   k_pool.stride(0), k_pool.stride(1), k_pool.stride(2),
                   v_pool.stride(0), v_pool.stride(1), v_pool.stride(2))


def decode_args(q, page_table, seq_lens, centroids=None, topk=0, bos=0, eos=0, sm_scale=1.0,
                order=None, status=None) -> DecodeArgs:
    _need(q, "q", torch.bfloat16, contiguous=True)
    _need(page_table, "page_table", torch.int32)
    _need(seq_lens, "seq_lens", torch.int32, contiguous=True)
    if page_table.dim() != 2 or page_table.stride(1) != 1:
        raise VtError(VT_ERR_INVALID_ARG, "page_table", "must be [B, max_pages] with unit inner stride")
    if centroids is not None:
        _need(centroids, "centroids", torch.float32, contiguous=True)
    if order is not None:
        _need(order, "order", torch.int32, contiguous=True)
    if status is not None:
        _need(status, "status", torch.int32)
    B, hq, _ = q.shape
    return DecodeArgs(B, hq, q.data_ptr(), page_table.data_ptr(), page_table.stride(0),
                      seq_lens.data_ptr(), _ptr(centroids), int(topk), int(bos), int(eos),
                      float(sm_scale), _ptr(order), _ptr(status))


def vt_build_centroids(k_pool: torch.Tensor, pages: torch.Tensor, centroids: torch.Tensor,
                       status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """centroids[p] = mean over the 16 tokens of K[p] for every physical page p in ``pages``."""
    lib = load_library()
    _need(pages, "pages", torch.int32, contiguous=True)
    _need(centroids, "centroids", torch.float32, contiguous=True)
    kv = paged_kv(k_pool, k_pool)
    rc = lib.vt_build_centroids(ctypes.byref(kv), pages.data_ptr(), pages.numel(),
                                centroids.data_ptr(), _ptr(status), _stream(k_pool))
    _check(rc, "vt_build_centroids")
    return centroids


def vt_select_pages(q, k_pool, v_pool, page_table, seq_lens, centroids, topk, bos, eos,
                    sel=None, n_sel=None, order=None, status=None, head_dim_v=None,
                    workspace=None):
    """Top-k page selection per (request, KV head).  Returns (sel [B,Hkv,kmax], n_sel [B,Hkv]).

    With ``workspace`` (from fused_workspace() for the same arguments) it calls
    vt_select_pages_ws (the persistent kernel, B <= 2048)."""
    lib = load_library()
    kv = paged_kv(k_pool, v_pool, head_dim_v)
    a = decode_args(q, page_table, seq_lens, centroids, topk, bos, eos, 1.0, order, status)
    kmax = topk + bos + eos
    B, hkv = q.shape[0], k_pool.shape[2]
    if sel is None:
        sel = torch.empty((B, hkv, kmax), dtype=torch.int32, device=q.device)
    if n_sel is None:
        n_sel = torch.empty((B, hkv), dtype=torch.int32, device=q.device)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, contiguous=True)
        rc = lib.vt_select_pages_ws(ctypes.byref(kv), ctypes.byref(a), sel.data_ptr(),
                                    n_sel.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                    _stream(q))
        _check(rc, "vt_select_pages_ws")
        return sel, n_sel
    rc = lib.vt_select_pages(ctypes.byref(kv), ctypes.byref(a), sel.data_ptr(), n_sel.data_ptr(),
                             _stream(q))
    _check(rc, "vt_select_pages")
    return sel, n_sel


def vt_select_pages_approx(q, k_pool, v_pool, page_table, seq_lens, centroids, topk, bos, eos,
                           seed, sel=None, n_sel=None, order=None, status=None, head_dim_v=None):
    """The indexer's lossy mode (one radix pass, seeded start in the last bin).  Returns
    (sel [B,Hkv,kmax], n_sel [B,Hkv])."""
    lib = load_library()
    kv = paged_kv(k_pool, v_pool, head_dim_v)
    a = decode_args(q, page_table, seq_lens, centroids, topk, bos, eos, 1.0, order, status)
    kmax = topk + bos + eos
    B, hkv = q.shape[0], k_pool.shape[2]
    if sel is None:
        sel = torch.empty((B, hkv, kmax), dtype=torch.int32, device=q.device)
    if n_sel is None:
        n_sel = torch.empty((B, hkv), dtype=torch.int32, device=q.device)
    rc = lib.vt_select_pages_approx(ctypes.byref(kv), ctypes.byref(a),
                                    ctypes.c_uint64(int(seed) & (2 ** 64 - 1)), sel.data_ptr(),
                                    n_sel.data_ptr(), _stream(q))
    _check(rc, "vt_select_pages_approx")
    return sel, n_sel


def vt_sparse_decode(q, k_pool, v_pool, page_table, seq_lens, sel, n_sel, sm_scale, out=None,
                     lse=None, status=None, head_dim_v=None, want_lse=True, workspace=None):
    """Attention over a given page selection.  Returns (out [B,Hq,Dv] bf16, lse [B,Hq] or None).

    With ``workspace`` (decode_workspace() for these arguments) it calls vt_sparse_decode_ws
    (the persistent kernel, B <= 2048)."""
    lib = load_library()
    kv = paged_kv(k_pool, v_pool, head_dim_v)
    kmax = sel.shape[2]
    a = decode_args(q, page_table, seq_lens, None, kmax, 0, 0, sm_scale, None, status)
    B, hq = q.shape[0], q.shape[1]
    if out is None:
        out = torch.empty((B, hq, kv.head_dim_v), dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, hq), dtype=torch.float32, device=q.device)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, contiguous=True)
        rc = lib.vt_sparse_decode_ws(ctypes.byref(kv), ctypes.byref(a), sel.data_ptr(),
                                     n_sel.data_ptr(), out.data_ptr(), _ptr(lse),
                                     workspace.data_ptr(), workspace.numel(), _stream(q))
        _check(rc, "vt_sparse_decode_ws")
        return out, lse
    rc = lib.vt_sparse_decode(ctypes.byref(kv), ctypes.byref(a), sel.data_ptr(), n_sel.data_ptr(),
                              out.data_ptr(), _ptr(lse), _stream(q))
    _check(rc, "vt_sparse_decode")
    return out, lse


def decode_workspace(q, k_pool, v_pool, page_table, seq_lens, sel, head_dim_v=None):
    """A zeroed workspace for vt_sparse_decode(..., workspace=) with these arguments (the
    decode call's arguments: kmax = sel.shape[2] selected pages, no centroids), or None."""
    lib = load_library()
    kv = paged_kv(k_pool, v_pool, head_dim_v)
    kmax = sel.shape[2]
    a = decode_args(q, page_table, seq_lens, None, kmax, 0, 0, 1.0, None, None)
    n = int(lib.vt_fused_workspace_size(ctypes.byref(kv), ctypes.byref(a)))
    return torch.zeros(n, dtype=torch.uint8, device=q.device) if n else None


def vt_fused_workspace_size(q, k_pool, v_pool, page_table, seq_lens, centroids, topk, bos, eos,
                            head_dim_v=None) -> int:
    """Bytes of workspace vt_sparse_decode_fused needs for these shapes (0 if none)."""
    lib = load_library()
    kv = paged_kv(k_pool, v_pool, head_dim_v)
    a = decode_args(q, page_table, seq_lens, centroids, topk, bos, eos, 1.0)
    return int(lib.vt_fused_workspace_size(ctypes.byref(kv), ctypes.byref(a)))


def fused_workspace(q, k_pool, v_pool, page_table, seq_lens, centroids, topk, bos, eos,
                    head_dim_v=None) -> Optional[torch.Tensor]:
    """A zero-filled workspace for vt_sparse_decode_fused (None when none is needed).

    Zero it once; every call leaves it ready for the next call with the same B * Hkv (zero it
    again before one with another B * Hkv).  Calls sharing one workspace must not overlap on
    the GPU.
    """
    n = vt_fused_workspace_size(q, k_pool, v_pool, page_table, seq_lens, centroids, topk, bos,
                                eos, head_dim_v)
    return torch.zeros(n, dtype=torch.uint8, device=q.device) if n else None


def vt_sparse_decode_fused(q, k_pool, v_pool, page_table, seq_lens, centroids, topk, bos, eos,
                           sm_scale, out=None, lse=None, sel=None, n_sel=None, order=None,
                           status=None, head_dim_v=None, want_lse=True, workspace=None):
    """Selection + attention in one call.  Returns (out, lse, sel, n_sel).

    ``workspace``: from fused_workspace(); allocated (zeroed) here when not given.
    """
    lib = load_library()
    kv = paged_kv(k_pool, v_pool, head_dim_v)
    a = decode_args(q, page_table, seq_lens, centroids, topk, bos, eos, sm_scale, order, status)
    B, hq = q.shape[0], q.shape[1]
    if out is None:
        out = torch.empty((B, hq, kv.head_dim_v), dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = int(lib.vt_fused_workspace_size(ctypes.byref(kv), ctypes.byref(a)))
        workspace = torch.zeros(n, dtype=torch.uint8, device=q.device) if n else None
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, contiguous=True)
    rc = lib.vt_sparse_decode_fused(ctypes.byref(kv), ctypes.byref(a), out.data_ptr(), _ptr(lse),
                                    _ptr(sel), _ptr(n_sel), _ptr(workspace),
                                    0 if workspace is None else workspace.numel(), _stream(q))
    _check(rc, "vt_sparse_decode_fused")
    return out, lse, sel, n_sel


def vt_sparse_decode_step(q, k_pool, v_pool, page_table, seq_lens, centroids, topk, bos, eos,
                          sm_scale, fill_pages, out=None, lse=None, sel=None, n_sel=None,
                          order=None, status=None, head_dim_v=None, want_lse=True,
                          workspace=None):
    """One step in one launch: the centroid build of fill_pages (int32, the pages filled at this
    step; written into ``centroids``) and the fused selection + attention.  Returns
    (out, lse, sel, n_sel)."""
    lib = load_library()
    kv = paged_kv(k_pool, v_pool, head_dim_v)
    a = decode_args(q, page_table, seq_lens, centroids, topk, bos, eos, sm_scale, order, status)
    _need(fill_pages, "fill_pages", torch.int32, contiguous=True)
    B, hq = q.shape[0], q.shape[1]
    if out is None:
        out = torch.empty((B, hq, kv.head_dim_v), dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = int(lib.vt_fused_workspace_size(ctypes.byref(kv), ctypes.byref(a)))
        workspace = torch.zeros(n, dtype=torch.uint8, device=q.device) if n else None
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, contiguous=True)
    rc = lib.vt_sparse_decode_step(ctypes.byref(kv), ctypes.byref(a), fill_pages.data_ptr(),
                                   fill_pages.numel(), centroids.data_ptr(), out.data_ptr(),
                                   _ptr(lse), _ptr(sel), _ptr(n_sel), _ptr(workspace),
                                   0 if workspace is None else workspace.numel(), _stream(q))
    _check(rc, "vt_sparse_decode_step")
    return out, lse, sel, n_sel


def vt_sparse_decode_fused_static(q, k_pool, v_pool, page_table, seq_lens, centroids, topk, bos,
                                  eos, sm_scale, out=None, lse=None, sel=None, n_sel=None,
                                  order=None, status=None, head_dim_v=None, want_lse=True):
    """vt_sparse_decode_fused on the library's own static scratch (no workspace argument).

    Calls on one device share that scratch: they must not overlap on the GPU.
    """
    lib = load_library()
    kv = paged_kv(k_pool, v_pool, head_dim_v)
    a = decode_args(q, page_table, seq_lens, centroids, topk, bos, eos, sm_scale, order, status)
    B, hq = q.shape[0], q.shape[1]
    if out is None:
        out = torch.empty((B, hq, kv.head_dim_v), dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, hq), dtype=torch.float32, device=q.device)
    rc = lib.vt_sparse_decode_fused_static(ctypes.byref(kv), ctypes.byref(a), out.data_ptr(),
                                           _ptr(lse), _ptr(sel), _ptr(n_sel), _stream(q))
    _check(rc, "vt_sparse_decode_fused_static")
    return out, lse, sel, n_sel


def vt_plan_requests(seq_lens: torch.Tensor, order: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Request order, longest (most pages) first; equal lengths keep index order."""
    lib = load_library()
    _need(seq_lens, "seq_lens", torch.int32, contiguous=True)
    if order is None:
        order = torch.empty_like(seq_lens)
    rc = lib.vt_plan_requests(seq_lens.data_ptr(), seq_lens.numel(), order.data_ptr(),
                              _stream(seq_lens))
    _check(rc, "vt_plan_requests")
    return order


# ---- dense attention and page calls -----------------------------------------------------------
# These run once per layer and step, often on little work, so their checks are written flat: one
# test per tensor, and the words for a failure only when there is one.

# (a torch built without CUDA has neither this nor the raw stream above; the package imports there)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_devices = [torch.device("cuda", i) for i in range(64)]


def _fail(t, name: str, dtype, dev: int, contiguous: bool = True):
    _need(t, name, dtype, contiguous=contiguous)
    raise VtError(VT_ERR_INVALID_ARG, name, f"on {t.device}, not on device {dev}")


def _vec(t, name: str, dtype, dev: int) -> int:
    """The address of a contiguous tensor of this type on device ``dev``."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev \
            or not t.is_contiguous():
        _fail(t, name, dtype, dev)
    return t.data_ptr()


def _sized(t: torch.Tensor, name: str, shape: tuple) -> None:
    if t.shape != shape:
        raise VtError(VT_ERR_INVALID_ARG, name, f"must be {list(shape)}, got {list(t.shape)}")


def _table(page_table: torch.Tensor, dev: int):
    """(rows, row stride, entries of a row) of a page table; what is between the rows of a view of
    some columns is not the table's."""
    if not isinstance(page_table, torch.Tensor) or page_table.dtype is not torch.int32 \
            or page_table.get_device() != dev:
        _fail(page_table, "page_table", torch.int32, dev, contiguous=False)
    st = page_table.stride()
    if len(st) != 2 or st[1] != 1:
        raise VtError(VT_ERR_INVALID_ARG, "page_table", "must be [B, max_pages] with unit inner stride")
    rows, width = page_table.shape
    stride = st[0] if rows > 1 else width
    return rows, stride, min(width, stride)


def _pools(k_pool, v_pool, dev: int) -> PagedKV:
    """paged_kv() of pools on device ``dev`` with the same pages and heads."""
    bf16 = torch.bfloat16
    if not (isinstance(k_pool, torch.Tensor) and isinstance(v_pool, torch.Tensor)) \
            or k_pool.dtype is not bf16 or v_pool.dtype is not bf16 \
            or k_pool.get_device() != dev or v_pool.get_device() != dev:
        paged_kv(k_pool, v_pool)
        raise VtError(VT_ERR_INVALID_ARG, "pools", f"not on device {dev}")
    ks, vs = k_pool.stride(), v_pool.stride()
    if len(ks) != 4 or len(vs) != 4 or ks[3] != 1 or vs[3] != 1:
        paged_kv(k_pool, v_pool)
    P, ps, hkv, d = k_pool.shape
    vp, vps, vh, dv = v_pool.shape
    if vp != P or vps != ps or vh != hkv:
        raise VtError(VT_ERR_INVALID_ARG, "pools", "K and V pools of different shapes")
    return PagedKV(k_pool.data_ptr(), v_pool.data_ptr(), P, ps, hkv, d, dv, ks[0], ks[1], ks[2],
                   vs[0], vs[1], vs[2])


def _status(status, dev: int):
    if status is None:
        return None
    if not isinstance(status, torch.Tensor) or status.dtype is not torch.int32 \
            or status.get_device() != dev:
        _fail(status, "status", torch.int32, dev, contiguous=False)
    return status.data_ptr()


def _gpu(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise VtError(VT_ERR_INVALID_ARG, name, "must be a CUDA tensor")
    return t.get_device()


def _prefill_args(q, k_pool, v_pool, page_table, seq_lens, q_start, sm_scale, status):
    dev = _gpu(q, "q")
    kv = _pools(k_pool, v_pool, dev)
    B, pt_stride, max_pages = _table(page_table, dev)
    if q.dtype is not torch.bfloat16:
        _need(q, "q", torch.bfloat16)
    if q.dim() != 3 or q.shape[2] != kv.head_dim:
        raise VtError(VT_ERR_INVALID_ARG, "q", f"must be [T, Hq, {kv.head_dim}]")
    T, hq, d = q.shape
    st, sh, sd = q.stride()
    if sd != 1 or (hq > 1 and sh != d):
        raise VtError(VT_ERR_INVALID_ARG, "q", "a token's heads must be contiguous")
    seq = _vec(seq_lens, "seq_lens", torch.int32, dev)
    start = _vec(q_start, "q_start", torch.int32, dev)
    _sized(seq_lens, "seq_lens", (B,))
    _sized(q_start, "q_start", (B + 1,))
    return kv, PrefillArgs(B, hq, T, q.data_ptr(), st if T > 1 else hq * d, start,
                           page_table.data_ptr(), pt_stride, seq, float(sm_scale),
                           _status(status, dev), max_pages)


def _attend_outputs(q, out, lse, want_lse):
    dev, shape = q.get_device(), q.shape
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _vec(out, "out", torch.bfloat16, dev)
        _sized(out, "out", shape)
    if lse is not None:
        _vec(lse, "lse", torch.float32, dev)
        _sized(lse, "lse", shape[:2])
    elif want_lse:
        lse = torch.empty_strided((shape[0], shape[1]), (shape[1], 1), dtype=torch.float32,
                                  device=q.device)
    return out, lse


def _workspace(workspace, need: int, dev: int):
    """(tensor, address, bytes) of the given workspace, or of a new one (any contents)."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=_devices[dev])
        return workspace, workspace.data_ptr(), need
    return workspace, _vec(workspace, "workspace", torch.uint8, dev), workspace.numel()


# What the C side decides by sizes and the binding relies on, so as not to ask at every call (held
# together by tests/test_workspace_rules.py): lists of up to LIST_SMEM rows grow without a
# workspace; prompts of PREFILL_SAME_WS tokens or more all need the same one.
LIST_SMEM = 2048
PREFILL_SAME_WS = 1024

# Bytes of workspace by what they depend on beside the device: a few shapes in a program's life.
_ws_bytes: dict = {}


def _ws_size(key: tuple, size_of) -> int:
    n = _ws_bytes.get(key)
    if n is None:
        n = int(size_of())
        if n:  # 0: the call has nothing to do, or will say what is wrong
            if len(_ws_bytes) >= 4096:
                _ws_bytes.clear()
            _ws_bytes[key] = n
    return n


def _device_call(fn, where: str, dev: int, *args) -> None:
    """fn(*args, stream) with device ``dev`` current (kernels run where their tensors are)."""
    if _current_device() == dev:
        rc = fn(*args, _raw_stream(dev) if _raw_stream is not None
                else torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    if rc != VT_OK:
        _check(rc, where)


def _prefill_ws(lib, dev: int, kv: PagedKV, a: PrefillArgs) -> int:
    if a.num_tokens < PREFILL_SAME_WS:
        return int(_on_device(dev, lib.vt_prefill_workspace_size, kv, a))
    return _ws_size(("prefill", dev, kv.head_dim),
                    lambda: _on_device(dev, lib.vt_prefill_workspace_size, kv, a))


def _on_device(dev: int, fn, *args):
    if _current_device() == dev:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def prefill_workspace(q, k_pool, v_pool, page_table, seq_lens, q_start) -> Optional[torch.Tensor]:
    """A workspace for vt_prefill with these shapes (any contents; None when none is needed)."""
    kv, a = _prefill_args(q, k_pool, v_pool, page_table, seq_lens, q_start, 1.0, None)
    dev = q.get_device()
    return _workspace(None, _prefill_ws(load_library(), dev, kv, a), dev)[0]


def vt_prefill(q, k_pool, v_pool, page_table, seq_lens, q_start, sm_scale, out=None, lse=None,
               status=None, want_lse=True, workspace=None):
    """Causal attention of packed prompts over the paged cache.  Returns (out, lse or None).

    ``q`` [T, Hq, D] (a view with another token stride is taken as it is): request b's rows are
    q_start[b] .. q_start[b+1], the last of its seq_lens[b] tokens.  Rows behind q_start[B] are
    left as they were.  ``workspace``: from prefill_workspace(); allocated here when not given.
    """
    lib = load_library()
    kv, a = _prefill_args(q, k_pool, v_pool, page_table, seq_lens, q_start, sm_scale, status)
    dev = q.get_device()
    out, lse = _attend_outputs(q, out, lse, want_lse)
    workspace, ws, ws_bytes = _workspace(workspace, _prefill_ws(lib, dev, kv, a), dev)
    _device_call(lib.vt_prefill, "vt_prefill", dev, kv, a, out.data_ptr(), _ptr(lse), ws, ws_bytes)
    return out, lse


def _shared_args(q, k_pool, v_pool, page_table, seq_lens, group_start, prefix_pages, sm_scale,
                 status):
    dev = _gpu(q, "q")
    kv = _pools(k_pool, v_pool, dev)
    B, pt_stride, max_pages = _table(page_table, dev)
    qp = _vec(q, "q", torch.bfloat16, dev)
    if q.dim() != 3 or q.shape[0] != B or q.shape[2] != kv.head_dim:
        raise VtError(VT_ERR_INVALID_ARG, "q", f"must be [{B}, Hq, {kv.head_dim}]")
    seq = _vec(seq_lens, "seq_lens", torch.int32, dev)
    start = _vec(group_start, "group_start", torch.int32, dev)
    prefix = _vec(prefix_pages, "prefix_pages", torch.int32, dev)
    groups = prefix_pages.numel()
    _sized(seq_lens, "seq_lens", (B,))
    _sized(group_start, "group_start", (groups + 1,))
    _sized(prefix_pages, "prefix_pages", (groups,))
    return kv, SharedPrefixArgs(B, q.shape[1], groups, qp, start, prefix, page_table.data_ptr(),
                                pt_stride, seq, float(sm_scale), _status(status, dev), max_pages)


def _shared_ws(lib, dev: int, kv: PagedKV, a: SharedPrefixArgs) -> int:
    if a.batch == 0 or a.num_groups == 0:
        return 0
    return _ws_size(("shared", dev, kv.head_dim, a.batch, a.num_q_heads, a.num_groups),
                    lambda: _on_device(dev, lib.vt_shared_prefix_workspace_size, kv, a))


def shared_prefix_workspace(q, k_pool, v_pool, page_table, seq_lens, group_start,
                            prefix_pages) -> Optional[torch.Tensor]:
    """A workspace for vt_shared_prefix_decode with these shapes (any contents)."""
    kv, a = _shared_args(q, k_pool, v_pool, page_table, seq_lens, group_start, prefix_pages, 1.0,
                         None)
    dev = q.get_device()
    return _workspace(None, _shared_ws(load_library(), dev, kv, a), dev)[0]


def vt_shared_prefix_decode(q, k_pool, v_pool, page_table, seq_lens, group_start, prefix_pages,
                            sm_scale, out=None, lse=None, status=None, want_lse=True,
                            workspace=None):
    """Decode attention over all pages of each request, where the requests group_start[g] ..
    group_start[g+1] share their first prefix_pages[g] pages, which are attended once for the
    group.  Returns (out [B, Hq, D], lse [B, Hq] or None).

    ``workspace``: from shared_prefix_workspace(); allocated here when not given.
    """
    lib = load_library()
    kv, a = _shared_args(q, k_pool, v_pool, page_table, seq_lens, group_start, prefix_pages,
                         sm_scale, status)
    dev = q.get_device()
    out, lse = _attend_outputs(q, out, lse, want_lse)
    workspace, ws, ws_bytes = _workspace(workspace, _shared_ws(lib, dev, kv, a), dev)
    _device_call(lib.vt_shared_prefix_decode, "vt_shared_prefix_decode", dev, kv, a,
                 out.data_ptr(), _ptr(lse), ws, ws_bytes)
    return out, lse


def _books(page_table, seq_lens, refs, status, dev: int) -> PageBooks:
    rows, pt_stride, max_pages = _table(page_table, dev)
    seq = _vec(seq_lens, "seq_lens", torch.int32, dev)
    _sized(seq_lens, "seq_lens", (rows,))
    return PageBooks(rows, page_table.data_ptr(), pt_stride, seq,
                     _vec(refs, "refs", torch.int32, dev), _status(status, dev), max_pages)


def _lists(dev: int, first, second, names: tuple):
    """(length, addresses) of one or two lists of equal length."""
    a = _vec(first, names[0], torch.int32, dev)
    if second is None:
        return first.numel(), a, None
    b = _vec(second, names[1], torch.int32, dev)
    if second.shape != first.shape:
        raise VtError(VT_ERR_INVALID_ARG, names[1], f"must be {list(first.shape)}, got "
                                                    f"{list(second.shape)}")
    return first.numel(), a, b


def _pool_books(k_pool, v_pool, refs, centroids, dev: int):
    kv = _pools(k_pool, v_pool, dev)
    if refs is not None and (not isinstance(refs, torch.Tensor) or refs.numel() != kv.num_pages):
        raise VtError(VT_ERR_INVALID_ARG, "refs", f"must be [{kv.num_pages}]")
    if centroids is None:
        return kv, None
    cent = _vec(centroids, "centroids", torch.float32, dev)
    _sized(centroids, "centroids", (kv.num_pages, kv.num_kv_heads, kv.head_dim))
    return kv, cent


def vt_copy_pages(k_pool, v_pool, src, dst, centroids=None, status=None) -> None:
    """Pages dst[i] become copies of pages src[i] (K, V and, where given, centroid rows); no page
    may be listed twice in ``dst``, or in both lists.  One pool as both K and V is copied once."""
    lib = load_library()
    dev = _gpu(k_pool, "k_pool")
    kv, cent = _pool_books(k_pool, v_pool, None, centroids, dev)
    n, a, b = _lists(dev, src, dst, ("src", "dst"))
    _device_call(lib.vt_copy_pages, "vt_copy_pages", dev, kv, a, b, n, cent, _status(status, dev))


def page_workspace(num_pages: int, n: int, device) -> torch.Tensor:
    """A workspace for the page calls: a pool of num_pages pages, lists of up to n requests."""
    return torch.empty(int(load_library().vt_page_workspace_size(int(num_pages), int(n))),
                       dtype=torch.uint8, device=device)


def _page_ws(lib, workspace, pages: int, n: int, dev: int):
    need = _ws_size(("pages", pages, n), lambda: lib.vt_page_workspace_size(pages, n)) \
        if workspace is None else 0
    return _workspace(workspace, need, dev)


def vt_fork_requests(k_pool, v_pool, page_table, seq_lens, refs, parents, children, status=None,
                     workspace=None) -> None:
    """Rows children[i] become forks of rows parents[i]: full pages are shared, a partly filled
    last page is copied to a page of its own (the lowest free ones, in list order)."""
    lib = load_library()
    dev = _gpu(k_pool, "k_pool")
    kv, _ = _pool_books(k_pool, v_pool, refs, None, dev)
    books = _books(page_table, seq_lens, refs, status, dev)
    n, a, b = _lists(dev, parents, children, ("parents", "children"))
    workspace, ws, ws_bytes = _page_ws(lib, workspace, kv.num_pages, n, dev)
    _device_call(lib.vt_fork_requests, "vt_fork_requests", dev, kv, books, a, b, n, ws, ws_bytes)


def vt_extend_requests(page_table, seq_lens, refs, requests, tokens, status=None,
                       workspace=None) -> None:
    """Rows requests[i] grow by tokens[i] tokens; the pages that takes are appended (the lowest
    free ones, in list order).  A new request starts from a row of length 0."""
    lib = load_library()
    dev = _gpu(refs, "refs")
    books = _books(page_table, seq_lens, refs, status, dev)
    n, a, b = _lists(dev, requests, tokens, ("requests", "tokens"))
    pages = refs.numel()
    ws, ws_bytes = None, 0
    if n > LIST_SMEM:
        workspace, ws, ws_bytes = _page_ws(lib, workspace, pages, n, dev)
    _device_call(lib.vt_extend_requests, "vt_extend_requests", dev, books, pages, a, b, n, ws,
                 ws_bytes)


def vt_free_requests(page_table, seq_lens, refs, requests, status=None) -> None:
    """Rows requests[i] end: their pages lose a reference, their lengths become 0."""
    lib = load_library()
    dev = _gpu(refs, "refs")
    books = _books(page_table, seq_lens, refs, status, dev)
    n, a, _ = _lists(dev, requests, None, ("requests",))
    _device_call(lib.vt_free_requests, "vt_free_requests", dev, books, refs.numel(), a, n)


def vt_compact_pages(k_pool, v_pool, page_table, seq_lens, refs, centroids=None, n_used=None,
                     status=None, workspace=None) -> torch.Tensor:
    """The used pages move to the front of the pools, tables and counts with them.  Returns
    n_used, int32 [1] on the device: pages n_used and up are free."""
    lib = load_library()
    dev = _gpu(k_pool, "k_pool")
    kv, cent = _pool_books(k_pool, v_pool, refs, centroids, dev)
    books = _books(page_table, seq_lens, refs, status, dev)
    if n_used is None:
        n_used = torch.empty_strided((1,), (1,), dtype=torch.int32, device=refs.device)
    workspace, ws, ws_bytes = _page_ws(lib, workspace, kv.num_pages, 0, dev)
    _device_call(lib.vt_compact_pages, "vt_compact_pages", dev, kv, books, cent,
                 _vec(n_used, "n_used", torch.int32, dev), ws, ws_bytes)
    return n_used


class PreparedCall:
    """One C entry point bound to fixed tensors: the arguments are checked and marshalled
    once, and each ``run()`` only launches (on the current stream).

    For a serving loop that calls the same operation on the same buffers every step (inputs
    refreshed in place, as with CUDA graphs).  The bound tensors must keep their storage,
    shapes and strides for the object's lifetime; it holds references to them.
    """

    def __init__(self, fn, args, device_index: int, where: str, keep, result):
        self._fn = fn
        self._args = args
        self._dev = device_index
        self._where = where
        self._keep = keep
        self.result = result

    def run(self):
        stream = _raw_stream(self._dev) if _raw_stream is not None else \
            torch.cuda.current_stream(self._dev).cuda_stream
        rc = self._fn(*self._args, stream)
        if rc != VT_OK:
            _check(rc, self._where)
        return self.result


def prepare_build_centroids(k_pool: torch.Tensor, pages: torch.Tensor, centroids: torch.Tensor,
                            status: Optional[torch.Tensor] = None) -> PreparedCall:
    """vt_build_centroids bound to these tensors; ``run()`` returns ``centroids``."""
    lib = load_library()
    _need(pages, "pages", torch.int32, contiguous=True)
    _need(centroids, "centroids", torch.float32, contiguous=True)
    if status is not None:
        _need(status, "status", torch.int32)
    kv = paged_kv(k_pool, k_pool)
    P = ctypes.c_void_p
    args = (ctypes.byref(kv), P(pages.data_ptr()), ctypes.c_int32(pages.numel()),
            P(centroids.data_ptr()), P(_ptr(status)))
    return PreparedCall(lib.vt_build_centroids, args, k_pool.get_device(), "vt_build_centroids",
                        (kv, k_pool, pages, centroids, status), centroids)


def prepare_sparse_decode_fused(q, k_pool, v_pool, page_table, seq_lens, centroids, topk, bos,
                                eos, sm_scale, out, lse=None, sel=None, n_sel=None, order=None,
                                status=None, head_dim_v=None, workspace=None) -> PreparedCall:
    """vt_sparse_decode_fused bound to these tensors; ``run()`` returns (out, lse, sel, n_sel).

    ``out`` (and ``lse`` if wanted) must be given; ``workspace`` as for the unprepared call
    (from fused_workspace(); required when the shapes need one).
    """
    lib = load_library()
    kv = paged_kv(k_pool, v_pool, head_dim_v)
    a = decode_args(q, page_table, seq_lens, centroids, topk, bos, eos, sm_scale, order, status)
    _need(out, "out", torch.bfloat16, contiguous=True)
    if lse is not None:
        _need(lse, "lse", torch.float32, contiguous=True)
    for t, name in ((sel, "sel"), (n_sel, "n_sel")):
        if t is not None:
            _need(t, name, torch.int32, contiguous=True)
    need = int(lib.vt_fused_workspace_size(ctypes.byref(kv), ctypes.byref(a)))
    if need:
        if workspace is None:
            raise VtError(VT_ERR_INVALID_ARG, "workspace", f"{need} bytes needed (fused_workspace())")
        _need(workspace, "workspace", torch.uint8, contiguous=True)
    P = ctypes.c_void_p
    args = (ctypes.byref(kv), ctypes.byref(a), P(out.data_ptr()), P(_ptr(lse)), P(_ptr(sel)),
            P(_ptr(n_sel)), P(_ptr(workspace)),
            ctypes.c_size_t(0 if workspace is None else workspace.numel()))
    keep = (kv, a, q, k_pool, v_pool, page_table, seq_lens, centroids, out, lse, sel, n_sel,
            order, status, workspace)
    return PreparedCall(lib.vt_sparse_decode_fused, args, q.get_device(), "vt_sparse_decode_fused",
                        keep, (out, lse, sel, n_sel))


def prepare_sparse_decode_step(q, k_pool, v_pool, page_table, seq_lens, centroids, topk, bos,
                               eos, sm_scale, fill_pages, out, lse=None, sel=None, n_sel=None,
                               order=None, status=None, head_dim_v=None,
                               workspace=None) -> PreparedCall:
    """vt_sparse_decode_step bound to these tensors (``fill_pages`` included: its contents may
    change between runs, its length may not); ``run()`` returns (out, lse, sel, n_sel)."""
    lib = load_library()
    fused = prepare_sparse_decode_fused(q, k_pool, v_pool, page_table, seq_lens, centroids, topk,
                                        bos, eos, sm_scale, out, lse, sel, n_sel, order, status,
                                        head_dim_v, workspace)
    _need(fill_pages, "fill_pages", torch.int32, contiguous=True)
    kv_ref, a_ref = fused._args[0], fused._args[1]
    P = ctypes.c_void_p
    args = (kv_ref, a_ref, P(fill_pages.data_ptr()), ctypes.c_int32(fill_pages.numel()),
            P(centroids.data_ptr())) + fused._args[2:]
    return PreparedCall(lib.vt_sparse_decode_step, args, q.get_device(), "vt_sparse_decode_step",
                        fused._keep + (fill_pages,), fused.result)


def _prepare_attend(lib, where: str, dev: int, kv, a, need: int, q, out, lse, workspace, keep):
    _vec(out, "out", torch.bfloat16, dev)
    _sized(out, "out", q.shape)
    if lse is not None:
        _vec(lse, "lse", torch.float32, dev)
        _sized(lse, "lse", q.shape[:2])
    if need and workspace is None:
        raise VtError(VT_ERR_INVALID_ARG, "workspace", f"{need} bytes needed (see {where})")
    ws = None if workspace is None else _vec(workspace, "workspace", torch.uint8, dev)
    P = ctypes.c_void_p
    args = (ctypes.byref(kv), ctypes.byref(a), P(out.data_ptr()), P(_ptr(lse)), P(ws),
            ctypes.c_size_t(0 if workspace is None else workspace.numel()))
    return PreparedCall(getattr(lib, where), args, dev, where,
                        (kv, a, q, out, lse, workspace) + keep, (out, lse))


def prepare_prefill(q, k_pool, v_pool, page_table, seq_lens, q_start, sm_scale, out, lse=None,
                    status=None, workspace=None) -> PreparedCall:
    """vt_prefill bound to these tensors (``q_start`` and ``seq_lens`` included: their contents may
    change between runs); ``run()`` returns (out, lse).  ``workspace``: from prefill_workspace();
    required when the shapes need one."""
    lib = load_library()
    kv, a = _prefill_args(q, k_pool, v_pool, page_table, seq_lens, q_start, sm_scale, status)
    dev = q.get_device()
    return _prepare_attend(lib, "vt_prefill", dev, kv, a, _prefill_ws(lib, dev, kv, a), q, out, lse,
                           workspace, (k_pool, v_pool, page_table, seq_lens, q_start, status))


def prepare_shared_prefix_decode(q, k_pool, v_pool, page_table, seq_lens, group_start,
                                 prefix_pages, sm_scale, out, lse=None, status=None,
                                 workspace=None) -> PreparedCall:
    """vt_shared_prefix_decode bound to these tensors; ``run()`` returns (out, lse).
    ``workspace``: from shared_prefix_workspace(); required when the shapes need one."""
    lib = load_library()
    kv, a = _shared_args(q, k_pool, v_pool, page_table, seq_lens, group_start, prefix_pages,
                         sm_scale, status)
    dev = q.get_device()
    return _prepare_attend(lib, "vt_shared_prefix_decode", dev, kv, a, _shared_ws(lib, dev, kv, a),
                           q, out, lse, workspace, (k_pool, v_pool, page_table, seq_lens,
                                                    group_start, prefix_pages, status))


def vt_abi_version() -> int:
    return int(load_library().vt_abi_version())
