"""Fused GQA flash-attention prefill for GB300 (sm_103a).

Thin ctypes binding over ``libgqa_prefill.so`` (the C ABI declared in
``include/gqa_prefill.h``): the functions here only marshal torch tensors into
pointers and sizes.  Every step of the computation runs in the CUDA kernels;
there is no CPU or PyTorch fallback, and calling in without the built library
raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

__all__ = ["load", "gqa_flash_prefill", "gqa_flash_prefill_debug", "prefill", "prepare",
           "PreparedCall",
           "plan", "force_block_n", "force_q_tiles", "get_device_status", "get_stream_status", "set_tuning",
           "gqa_flash_prefill_splitkv", "splitkv_workspace", "prefill_splitkv",
           "gqa_flash_prefill_splitkv_noalloc", "prefill_splitkv_noalloc",
           "gqa_flash_prefill_masked", "prefill_masked",
           "NOALLOC_SCRATCH_BYTES", "gqa_flash_prefill_paged", "prefill_paged",
           "clear_config_cache", "config_block_n", "selftest_timeout", "GQAError",
           "GQA_F16", "GQA_BF16", "GQA_DEV_TIMEOUT", "GQA_DEV_BAD_METADATA", "SPLITS_BALANCED",
           "FLAG_METADATA_READY", "set_call_flags", "get_call_flags",
           "GQA_CACHE_16", "GQA_CACHE_E4M3", "Rope", "gqa_rope", "gqa_cache_write",
           "gqa_cache_read", "gqa_cache_attention", "cache_attention_workspace",
           "prepare_call", "PreparedOp", "cache_write", "cache_read", "cache_attention",
           "gqa_prefill_backward", "prefill_backward_workspace", "prefill_backward",
           "gqa_rms_norm", "rms_norm", "gqa_rms_norm_backward", "rms_norm_backward_workspace",
           "rms_norm_backward", "GQA_F32",
           "EXPORTED_SYMBOLS"]

GQA_F16, GQA_BF16, GQA_F32 = 0, 1, 2  # GQA_F32: residual streams and weights of the norm only
GQA_OK, GQA_ERR_INVALID, GQA_ERR_UNSUPPORTED, GQA_ERR_CUDA = 0, -1, -2, -3
GQA_DEV_TIMEOUT, GQA_DEV_BAD_METADATA = 1, 2
SPLITS_BALANCED = -1  # num_splits of the balanced split (GQA_SPLITS_BALANCED)
FLAG_METADATA_READY = 1  # GQA_FLAG_METADATA_READY (gqa_prefill_set_call_flags)
GQA_CACHE_16, GQA_CACHE_E4M3 = 0, 1  # element type of a page pool

EXPORTED_SYMBOLS = [
    "gqa_flash_prefill", "gqa_flash_prefill_debug", "gqa_prefill_plan",
    "gqa_prefill_force_block_n", "gqa_prefill_get_device_status",
    "gqa_prefill_status_string", "gqa_prefill_version", "gqa_prefill_set_tuning",
    "gqa_prefill_clear_config_cache", "gqa_prefill_config_block_n",
    "gqa_prefill_selftest_timeout", "gqa_prefill_force_q_tiles",
    "gqa_flash_prefill_splitkv", "gqa_prefill_splitkv_workspace",
    "gqa_flash_prefill_splitkv_noalloc", "gqa_flash_prefill_paged",
    "gqa_prefill_get_stream_status", "gqa_flash_prefill_masked",
    "gqa_prefill_set_call_flags", "gqa_prefill_get_call_flags",
    "gqa_rope", "gqa_cache_write", "gqa_cache_read", "gqa_cache_attention",
    "gqa_cache_attention_workspace", "gqa_prefill_backward", "gqa_prefill_backward_workspace",
    "gqa_rms_norm", "gqa_rms_norm_backward", "gqa_rms_norm_backward_workspace",
]
NOALLOC_SCRATCH_BYTES = 32 << 20  # the library's file-scope split-KV scratch (gqa_prefill.h)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgqa_prefill.so")
_lib = None


class GQAError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {code} ({_status_string(code)})")


class _Plan(ctypes.Structure):
    _fields_ = [("rows_per_unit", ctypes.c_int), ("block_n", ctypes.c_int),
                ("kv_stages", ctypes.c_int), ("ctas_per_sm", ctypes.c_int),
                ("grid", ctypes.c_int), ("max_units", ctypes.c_int),
                ("q_tiles", ctypes.c_int)]


class _RopeArgs(ctypes.Structure):  # gqa_rope_t
    _fields_ = [("positions", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p),
                ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("inverse", ctypes.c_int), ("attn_factor", ctypes.c_float),
                ("Hq", ctypes.c_int), ("q", ctypes.c_void_p), ("q_stride", ctypes.c_longlong),
                ("q_out", ctypes.c_void_p), ("q_out_stride", ctypes.c_longlong)]


def load(path: Optional[str] = None):
    """Load libgqa_prefill.so (built by ``__graft_entry__.build()`` or
    ``python -m gqa_flash_attention_prefill_gb300.build``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    # GQA_PREFILL_LIB names another build of the same library (used to time
    # two builds against each other on one machine).
    p = path or os.environ.get("GQA_PREFILL_LIB") or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"CUDA library {p} is missing: build it with "
            "`python -m gqa_flash_attention_prefill_gb300.build`")
    lib = ctypes.CDLL(p)
    vp, i32p, fp = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
    core = [vp, vp, vp, i32p, i32p, i32p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
            ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
            ctypes.c_float, ctypes.c_int, fp, ctypes.c_int, vp, fp, vp]
    lib.gqa_flash_prefill.argtypes = core
    lib.gqa_flash_prefill.restype = ctypes.c_int
    lib.gqa_flash_prefill_debug.argtypes = core + [vp]
    lib.gqa_flash_prefill_debug.restype = ctypes.c_int
    lib.gqa_flash_prefill_splitkv.argtypes = core[:-1] + [ctypes.c_int, vp, ctypes.c_size_t, vp]
    lib.gqa_flash_prefill_splitkv.restype = ctypes.c_int
    lib.gqa_flash_prefill_masked.argtypes = core[:18] + [vp, vp, ctypes.c_longlong, vp, fp, vp]
    lib.gqa_flash_prefill_masked.restype = ctypes.c_int
    lib.gqa_flash_prefill_paged.argtypes = [vp] * 7 + [ctypes.c_int] * 10 + [
        ctypes.c_float, ctypes.c_int, vp, ctypes.c_int, vp, vp, vp]
    lib.gqa_flash_prefill_paged.restype = ctypes.c_int
    lib.gqa_flash_prefill_splitkv_noalloc.argtypes = core[:-1] + [ctypes.c_int, vp]
    lib.gqa_flash_prefill_splitkv_noalloc.restype = ctypes.c_int
    lib.gqa_prefill_splitkv_workspace.argtypes = [ctypes.c_int] * 9 + [
        ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_size_t)]
    lib.gqa_prefill_splitkv_workspace.restype = ctypes.c_int
    lib.gqa_prefill_plan.argtypes = [ctypes.c_int] * 8 + [ctypes.POINTER(_Plan)]
    lib.gqa_prefill_plan.restype = ctypes.c_int
    lib.gqa_prefill_force_block_n.argtypes = [ctypes.c_int]
    lib.gqa_prefill_force_block_n.restype = ctypes.c_int
    lib.gqa_prefill_force_q_tiles.argtypes = [ctypes.c_int]
    lib.gqa_prefill_force_q_tiles.restype = ctypes.c_int
    lib.gqa_prefill_get_device_status.argtypes = [ctypes.POINTER(ctypes.c_int)]
    lib.gqa_prefill_get_device_status.restype = ctypes.c_int
    lib.gqa_prefill_get_stream_status.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int)]
    lib.gqa_prefill_get_stream_status.restype = ctypes.c_int
    lib.gqa_prefill_status_string.argtypes = [ctypes.c_int]
    lib.gqa_prefill_status_string.restype = ctypes.c_char_p
    lib.gqa_prefill_version.argtypes = []
    lib.gqa_prefill_version.restype = ctypes.c_char_p
    lib.gqa_prefill_set_tuning.argtypes = [ctypes.c_int]
    lib.gqa_prefill_set_tuning.restype = ctypes.c_int
    lib.gqa_prefill_clear_config_cache.argtypes = []
    lib.gqa_prefill_clear_config_cache.restype = ctypes.c_int
    lib.gqa_prefill_config_block_n.argtypes = [ctypes.c_int] * 7 + [
        ctypes.POINTER(ctypes.c_int)] * 3
    lib.gqa_prefill_config_block_n.restype = ctypes.c_int
    lib.gqa_prefill_selftest_timeout.argtypes = [ctypes.c_int, ctypes.c_void_p,
                                                 ctypes.POINTER(ctypes.c_int)]
    lib.gqa_prefill_selftest_timeout.restype = ctypes.c_int
    lib.gqa_prefill_set_call_flags.argtypes = [ctypes.c_uint]
    lib.gqa_prefill_set_call_flags.restype = ctypes.c_int
    lib.gqa_prefill_get_call_flags.argtypes = []
    lib.gqa_prefill_get_call_flags.restype = ctypes.c_uint
    i, ll = ctypes.c_int, ctypes.c_longlong
    lib.gqa_rope.argtypes = [ctypes.POINTER(_RopeArgs), vp, ll, vp, ll, i, i, i, i, vp]
    lib.gqa_cache_write.argtypes = [vp, ll, vp, ll] + [vp] * 4 + [i] * 9 + [vp] * 4 + [
        ctypes.POINTER(_RopeArgs), vp]
    lib.gqa_cache_read.argtypes = [vp] * 4 + [i, vp, vp] + [i] * 3 + [vp, vp] + [i] * 5 + [vp] * 3
    lib.gqa_cache_attention.argtypes = [vp] * 5 + [i] + [vp] * 4 + [i] * 10 + [
        ctypes.c_float, i, vp, i, vp, vp, ll, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.gqa_cache_attention_workspace.argtypes = [i] * 8 + [ctypes.POINTER(ctypes.c_size_t)]
    lib.gqa_prefill_backward.argtypes = [vp] * 6 + [i] * 7 + [ctypes.c_float, i] + [vp] * 10 + [
        ctypes.c_size_t, vp]
    lib.gqa_prefill_backward_workspace.argtypes = [i] * 7 + [ctypes.POINTER(ctypes.c_size_t)]
    lib.gqa_rms_norm.argtypes = [vp, ll, vp, vp, i, vp, i, ctypes.c_float, ctypes.c_float] + [i] * 6 + [
        vp, ll, vp, vp, vp]
    lib.gqa_rms_norm_backward.argtypes = [vp, ll, vp, ll, i, vp, vp, i, ctypes.c_float, vp] + [i] * 4 + [
        vp, ll, vp, vp, vp, ctypes.c_size_t, vp]
    lib.gqa_rms_norm_backward_workspace.argtypes = [i] * 4 + [ctypes.POINTER(ctypes.c_size_t)]
    for f in (lib.gqa_rope, lib.gqa_cache_write, lib.gqa_cache_read, lib.gqa_cache_attention,
              lib.gqa_cache_attention_workspace, lib.gqa_prefill_backward,
              lib.gqa_prefill_backward_workspace, lib.gqa_rms_norm, lib.gqa_rms_norm_backward,
              lib.gqa_rms_norm_backward_workspace):
        f.restype = i
    if path is None:
        _lib = lib
    return lib


def _status_string(code: int) -> str:
    try:
        return load().gqa_prefill_status_string(code).decode()
    except Exception:  # pragma: no cover - library missing
        return "?"


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return GQA_BF16
    if t.dtype == torch.float16:
        return GQA_F16
    raise TypeError(f"q/k/v must be float16 or bfloat16, got {t.dtype}")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_handle(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _allocating(stream):
    """Context in which torch allocates for `stream`: the allocator hands a
    freed block to the next allocation of the stream it was made on, so memory
    that only a call on another stream uses has to be made on that one."""
    import contextlib
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        # Handles 0 and 1 are the legacy default stream; torch takes 0 for "a new one".
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _result(shape, dtype, device, stream):
    """A new tensor that a call on `stream` fills and the caller's current
    stream may read: once freed, its block waits for both."""
    import torch
    with _allocating(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream())
    return t


def _outputs(q, out, lse, with_lse, stream):
    """(out, lse) of a call on `stream`, new where not given."""
    import torch
    if out is None:
        out = _result(q.shape, q.dtype, q.device, stream)
    if lse is None and with_lse:
        lse = _result(q.shape[:2], torch.float32, q.device, stream)
    return out, lse


def _args(q, k, v, cu_seqlens_q, prefix_lens, kv_indptr, scale, window, sinks,
          smooth_softmax, out, lse, stream, max_seqlen_q):
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        if t.dim() != 3 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [rows, heads, d] tensor")
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("prefix_lens", prefix_lens),
                    ("kv_indptr", kv_indptr)):
        if str(t.dtype) != "torch.int32" or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor")
    total_q, hq, d = q.shape
    total_kv, hkv, _ = k.shape
    return (_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens_q), _ptr(prefix_lens),
            _ptr(kv_indptr), int(prefix_lens.numel()), int(total_q), int(total_kv),
            int(max_seqlen_q), int(hq), int(hkv), int(d), _dtype_code(q), float(scale),
            int(window), _ptr(sinks), 1 if smooth_softmax else 0, _ptr(out), _ptr(lse),
            _stream_handle(stream))


def gqa_flash_prefill(q, k, v, cu_seqlens_q, prefix_lens, kv_indptr, scale,
                      window=0, sinks=None, smooth_softmax=False, out=None,
                      lse=None, stream=None, max_seqlen_q=0):
    """Marshal torch CUDA tensors into the C ABI call (see gqa_prefill.h).
    ``out`` [total_q, Hq, d] and ``lse`` (fp32 [total_q, Hq] or None) are
    written in place; returns ``out``."""
    rc = load().gqa_flash_prefill(*_args(q, k, v, cu_seqlens_q, prefix_lens,
                                         kv_indptr, scale, window, sinks,
                                         smooth_softmax, out, lse, stream,
                                         max_seqlen_q))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_flash_prefill")
    return out


def gqa_flash_prefill_masked(q, k, v, cu_seqlens_q, prefix_lens, kv_indptr, scale,
                             custom_mask, mask_indptr, window=0, sinks=None,
                             smooth_softmax=False, out=None, lse=None, stream=None,
                             max_seqlen_q=0):
    """gqa_flash_prefill with a custom mask (see gqa_prefill.h): custom_mask
    is a device tensor of 32-bit words (int32 or uint32), mask_indptr a
    device int32 [B+1] of word offsets."""
    for name, t in (("custom_mask", custom_mask), ("mask_indptr", mask_indptr)):
        if t.element_size() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor of 32-bit words")
    a = _args(q, k, v, cu_seqlens_q, prefix_lens, kv_indptr, scale, window, sinks,
              smooth_softmax, out, lse, stream, max_seqlen_q)
    rc = load().gqa_flash_prefill_masked(*a[:18], _ptr(custom_mask), _ptr(mask_indptr),
                                         int(custom_mask.numel()), *a[18:])
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_flash_prefill_masked")
    return out


def prefill_masked(batch, custom_mask, mask_indptr, out=None, lse=None, with_lse=True,
                   stream=None):
    """gqa_flash_prefill_masked on one ``workloads.Batch`` already on the GPU
    (custom_mask / mask_indptr from ``workloads.pack_custom_mask``, on the
    GPU); allocates out/lse with torch when not given.  Returns (out, lse)."""
    out, lse = _outputs(batch.q, out, lse, with_lse, stream)
    gqa_flash_prefill_masked(batch.q, batch.k, batch.v, batch.cu_seqlens_q, batch.prefix_lens,
                             batch.kv_indptr, batch.scale, custom_mask, mask_indptr,
                             window=batch.window, sinks=batch.sinks, smooth_softmax=batch.smooth,
                             out=out, lse=lse, stream=stream, max_seqlen_q=batch.max_seqlen_q)
    return out, lse


def gqa_flash_prefill_debug(q, k, v, cu_seqlens_q, prefix_lens, kv_indptr, scale,
                            unit_log, window=0, sinks=None, smooth_softmax=False,
                            out=None, lse=None, stream=None, max_seqlen_q=0):
    """Same as gqa_flash_prefill, and writes one 8-int record per work unit
    into ``unit_log`` (device int32 [max_units, 8])."""
    rc = load().gqa_flash_prefill_debug(*_args(q, k, v, cu_seqlens_q, prefix_lens,
                                               kv_indptr, scale, window, sinks,
                                               smooth_softmax, out, lse, stream,
                                               max_seqlen_q), _ptr(unit_log))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_flash_prefill_debug")
    return out


def gqa_flash_prefill_splitkv(q, k, v, cu_seqlens_q, prefix_lens, kv_indptr, scale,
                              workspace, num_splits=0, window=0, sinks=None,
                              smooth_softmax=False, out=None, lse=None, stream=None,
                              max_seqlen_q=0):
    """Split-KV form of gqa_flash_prefill (see gqa_prefill.h); ``workspace``
    is a device tensor (any dtype) at least ``splitkv_workspace(...)`` bytes,
    or None when the call does not split."""
    a = _args(q, k, v, cu_seqlens_q, prefix_lens, kv_indptr, scale, window, sinks,
              smooth_softmax, out, lse, stream, max_seqlen_q)
    ws = _ptr(workspace)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().gqa_flash_prefill_splitkv(*a[:-1], int(num_splits), ws, nbytes, a[-1])
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_flash_prefill_splitkv")
    return out


def splitkv_workspace(num_seqs, total_q, max_seqlen_q, hq, hkv, d, dtype, window,
                      num_splits=0):
    """(splits used, workspace bytes) for a split-KV call with these shapes."""
    used, nbytes = ctypes.c_int(0), ctypes.c_size_t(0)
    code = dtype if isinstance(dtype, int) else (GQA_BF16 if "bf16" in str(dtype) else GQA_F16)
    rc = load().gqa_prefill_splitkv_workspace(int(num_seqs), int(total_q), int(max_seqlen_q),
                                              int(hq), int(hkv), int(d), code, int(window),
                                              int(num_splits), ctypes.byref(used),
                                              ctypes.byref(nbytes))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_prefill_splitkv_workspace")
    return used.value, nbytes.value


def gqa_flash_prefill_splitkv_noalloc(q, k, v, cu_seqlens_q, prefix_lens, kv_indptr, scale,
                                      num_splits=0, window=0, sinks=None, smooth_softmax=False,
                                      out=None, lse=None, stream=None, max_seqlen_q=0):
    """Split-KV with the library's file-scope scratch (see gqa_prefill.h): no
    workspace, nothing allocated; overlapping calls race on the scratch."""
    a = _args(q, k, v, cu_seqlens_q, prefix_lens, kv_indptr, scale, window, sinks,
              smooth_softmax, out, lse, stream, max_seqlen_q)
    rc = load().gqa_flash_prefill_splitkv_noalloc(*a[:-1], int(num_splits), a[-1])
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_flash_prefill_splitkv_noalloc")
    return out


def prefill_splitkv_noalloc(batch, num_splits=0, out=None, lse=None, stream=None):
    """gqa_flash_prefill_splitkv_noalloc on one ``workloads.Batch`` already on
    the GPU, into caller buffers (out is required: the call allocates nothing)."""
    gqa_flash_prefill_splitkv_noalloc(batch.q, batch.k, batch.v, batch.cu_seqlens_q,
                                      batch.prefix_lens, batch.kv_indptr, batch.scale,
                                      num_splits=num_splits, window=batch.window,
                                      sinks=batch.sinks, smooth_softmax=batch.smooth, out=out,
                                      lse=lse, stream=stream, max_seqlen_q=batch.max_seqlen_q)
    return out, lse


def prefill_splitkv(batch, num_splits=0, workspace=None, out=None, lse=None, with_lse=True,
                    stream=None):
    """Split-KV run of one ``workloads.Batch`` already on the GPU; allocates the
    workspace (and out/lse) with torch when not given.  Returns (out, lse)."""
    import torch
    out, lse = _outputs(batch.q, out, lse, with_lse, stream)
    used, nbytes = splitkv_workspace(batch.num_seqs, batch.total_q, batch.max_seqlen_q,
                                     batch.hq, batch.hkv, batch.d, batch.dtype_name,
                                     batch.window, num_splits)
    if workspace is None and nbytes > 0:
        with _allocating(stream):
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=batch.q.device)
    gqa_flash_prefill_splitkv(batch.q, batch.k, batch.v, batch.cu_seqlens_q,
                              batch.prefix_lens, batch.kv_indptr, batch.scale, workspace,
                              num_splits=num_splits, window=batch.window, sinks=batch.sinks,
                              smooth_softmax=batch.smooth, out=out, lse=lse, stream=stream,
                              max_seqlen_q=batch.max_seqlen_q)
    return out, lse


def gqa_flash_prefill_paged(q, k_pages, v_pages, cu_seqlens_q, prefix_lens, kv_page_indptr,
                            kv_page_indices, scale, window=0, sinks=None, smooth_softmax=False,
                            out=None, lse=None, stream=None, max_seqlen_q=0):
    """Marshal a paged-KV call (see gqa_prefill.h): k_pages / v_pages are
    [num_pages, page_size, Hkv, d]; returns ``out``."""
    for name, t in (("q", q), ("out", out)):
        if t.dim() != 3 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [rows, heads, d] tensor")
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [pages, page_size, heads, d] tensor")
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("prefix_lens", prefix_lens),
                    ("kv_page_indptr", kv_page_indptr), ("kv_page_indices", kv_page_indices)):
        if str(t.dtype) != "torch.int32" or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor")
    total_q, hq, d = q.shape
    num_pages, page_size, hkv, _ = k_pages.shape
    rc = load().gqa_flash_prefill_paged(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(cu_seqlens_q), _ptr(prefix_lens),
        _ptr(kv_page_indptr), _ptr(kv_page_indices), int(kv_page_indices.numel()),
        int(page_size), int(num_pages), int(prefix_lens.numel()), int(total_q),
        int(max_seqlen_q), int(hq), int(hkv), int(d), _dtype_code(q), float(scale), int(window),
        _ptr(sinks), 1 if smooth_softmax else 0, _ptr(out), _ptr(lse), _stream_handle(stream))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_flash_prefill_paged")
    return out


def prefill_paged(paged, out=None, lse=None, with_lse=True, stream=None):
    """Run one ``workloads.PagedBatch`` already on the GPU.  Returns (out, lse)."""
    b = paged.batch
    out, lse = _outputs(b.q, out, lse, with_lse, stream)
    gqa_flash_prefill_paged(b.q, paged.k_pages, paged.v_pages, b.cu_seqlens_q, b.prefix_lens,
                            paged.page_indptr, paged.page_indices, b.scale, window=b.window,
                            sinks=b.sinks, smooth_softmax=b.smooth, out=out, lse=lse,
                            stream=stream, max_seqlen_q=b.max_seqlen_q)
    return out, lse


def prefill(batch, out=None, lse=None, with_lse=True, stream=None):
    """Run one ``workloads.Batch`` already on the GPU; allocates out/lse with
    torch when not given.  Returns (out, lse)."""
    out, lse = _outputs(batch.q, out, lse, with_lse, stream)
    gqa_flash_prefill(batch.q, batch.k, batch.v, batch.cu_seqlens_q,
                      batch.prefix_lens, batch.kv_indptr, batch.scale,
                      window=batch.window, sinks=batch.sinks,
                      smooth_softmax=batch.smooth, out=out, lse=lse,
                      stream=stream, max_seqlen_q=batch.max_seqlen_q)
    return out, lse


class PreparedCall:
    """gqa_flash_prefill (or, with ``num_splits``, gqa_flash_prefill_splitkv
    on ``workspace``) with its arguments marshalled once: calling the object
    re-issues the same C ABI call (same buffers, same stream), which keeps
    the host cost of a call to the ctypes round trip.  For callers that
    replay a fixed sequence of calls over resident buffers, such as the
    layers of a prefill."""

    __slots__ = ("_fn", "_args", "_name", "out", "lse", "workspace")

    def __init__(self, batch, out, lse=None, stream=None, num_splits=None, workspace=None):
        a = _args(batch.q, batch.k, batch.v, batch.cu_seqlens_q, batch.prefix_lens,
                  batch.kv_indptr, batch.scale, batch.window, batch.sinks, batch.smooth, out, lse,
                  stream, batch.max_seqlen_q)
        if num_splits is None:
            self._fn, self._name, self._args = load().gqa_flash_prefill, "gqa_flash_prefill", a
        else:
            nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
            self._fn, self._name = load().gqa_flash_prefill_splitkv, "gqa_flash_prefill_splitkv"
            self._args = a[:-1] + (int(num_splits), _ptr(workspace), nbytes, a[-1])
        self.out, self.lse, self.workspace = out, lse, workspace

    def __call__(self):
        rc = self._fn(*self._args)
        if rc != GQA_OK:
            raise GQAError(rc, self._name)


def prepare(batch, out, lse=None, stream=None, num_splits=None, workspace=None) -> PreparedCall:
    """A PreparedCall of one ``workloads.Batch`` already on the GPU, writing
    ``out`` (and ``lse`` when given) on ``stream``; with ``num_splits`` (for
    example SPLITS_BALANCED) the split-KV entry point on ``workspace``."""
    return PreparedCall(batch, out, lse, stream, num_splits, workspace)


# ------------------------------------------------------- the paged cache's operators
class PreparedOp:
    """One C ABI call with its arguments marshalled: calling the object issues
    it again (same buffers, same stream, on the device that was current when it
    was made, which has to be current again).  Made by :func:`prepare_call`;
    holds the tensors it points to."""

    __slots__ = ("_fn", "_args", "_name", "_keep", "_current", "_device")

    def __init__(self, fn, args, name, keep):
        import torch
        self._fn, self._args, self._name, self._keep = fn, args, name, keep
        self._current = torch.cuda.current_device
        # Asked at every call only where there is another device: it takes 1 us.
        self._device = self._current() if torch.cuda.device_count() > 1 else None

    def __call__(self):
        if self._device is not None and self._current() != self._device:
            raise ValueError(f"{self._name} was prepared on cuda:{self._device}, which is not the "
                             "current device")
        rc = self._fn(*self._args)
        if rc != GQA_OK:
            raise GQAError(rc, self._name)


def prepare_call(function, *args, **kwargs) -> PreparedOp:
    """The call ``function(*args, **kwargs)`` marshalled once, to be issued by
    calling the result.  For gqa_rope, gqa_cache_write, gqa_cache_read,
    gqa_cache_attention, gqa_prefill_backward, gqa_rms_norm and
    gqa_rms_norm_backward."""
    marshal = _MARSHAL.get(function)
    if marshal is None:
        raise ValueError("prepare_call takes gqa_rope, gqa_cache_write, gqa_cache_read, "
                         "gqa_cache_attention, gqa_prefill_backward, gqa_rms_norm or "
                         "gqa_rms_norm_backward")
    return marshal(*args, **kwargs)


def _on_device(**tensors):
    """Every given tensor is a CUDA tensor of the current device: the library
    launches there, and a pointer of another device would fault."""
    import torch
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.device.index != torch.cuda.current_device():
            raise ValueError(f"{name} is on {t.device}, not on the current device")


def _int32(**tensors):
    for name, t in tensors.items():
        if t is not None and (str(t.dtype) != "torch.int32" or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous int32 tensor")


def _rows(name, t, like=None):
    """Rows [rows, heads, d] whose heads are packed: returns the row stride."""
    if t.dim() != 3 or t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise ValueError(f"{name} must be [rows, heads, d] with packed heads")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype):
        raise ValueError(f"{name} must have the shape and type of its input")
    # The stride of a single row is never used; torch may report any.
    return int(t.stride(0)) if t.shape[0] > 1 else int(t.shape[1] * t.shape[2])


def _pool(k_pages, v_pages, k_scales, v_scales, dtype=None):
    """(cache type, pages, page size, heads, d) of a checked page pool."""
    import torch
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [pages, page_size, heads, d] tensor")
    if k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype:
        raise ValueError("k_pages and v_pages must agree in shape and type")
    shape = [int(n) for n in k_pages.shape]
    if k_pages.dtype in (torch.float16, torch.bfloat16):
        if k_scales is not None or v_scales is not None:
            raise ValueError("a 16-bit page pool has no scales")
        if dtype is not None and k_pages.dtype != dtype:
            raise TypeError(f"a 16-bit page pool must have the type of the rows, {dtype}")
        return (GQA_CACHE_16, *shape)
    if k_pages.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError(f"pages must be float16, bfloat16 or e4m3, got {k_pages.dtype}")
    for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        if t is None or t.element_size() != 1 or list(t.shape) != shape[:3] or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous byte tensor [pages, page_size, heads]")
    return (GQA_CACHE_E4M3, *shape)


def _lengths(cu_seqlens_q, prefix_lens, kv_page_indptr):
    n = int(prefix_lens.numel())
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("kv_page_indptr", kv_page_indptr)):
        if t.numel() != n + 1:
            raise ValueError(f"{name} must have one entry more than prefix_lens")
    return n


class Rope:
    """Rotary positions (gqa_rope_t): ``inv_freq`` fp64 [rot_dim / 2] on the
    GPU, the pair order, the factor on rotated values, and, in
    gqa_cache_write, the query rows to rotate on the way (``q`` into
    ``q_out``) and explicit ``positions`` (int32, else the keys' own)."""

    def __init__(self, inv_freq, positions=None, interleaved=False, attn_factor=1.0, q=None,
                 q_out=None, inverse=False):
        import torch
        if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous float64 vector")
        if (q is None) != (q_out is None):
            raise ValueError("q and q_out go together")
        _int32(positions=positions)
        self.inv_freq, self.positions, self.interleaved = inv_freq, positions, bool(interleaved)
        self.attn_factor, self.q, self.q_out = float(attn_factor), q, q_out
        self.inverse = bool(inverse)

    def _args(self, rows, dtype, d):
        _on_device(inv_freq=self.inv_freq, positions=self.positions, q=self.q, q_out=self.q_out)
        if self.positions is not None and self.positions.numel() != rows:
            raise ValueError("positions must have one entry per row")
        a = _RopeArgs(_ptr(self.positions), _ptr(self.inv_freq), 2 * self.inv_freq.numel(),
                      int(self.interleaved), int(self.inverse), self.attn_factor, 0, None, 0, None, 0)
        if self.q is not None:
            qs, os_ = _rows("q", self.q), _rows("q_out", self.q_out, self.q)
            if self.q.shape[0] != rows or self.q.shape[2] != d or self.q.dtype != dtype:
                raise ValueError("q must have as many rows as k, its head dim and its type")
            a.Hq, a.q, a.q_stride = int(self.q.shape[1]), _ptr(self.q), qs
            a.q_out, a.q_out_stride = _ptr(self.q_out), os_
        return a


def _marshal_rope(q, positions, inv_freq, out, k=None, k_out=None, interleaved=False,
                  attn_factor=1.0, inverse=False, stream=None):
    if positions is None or (k is None) != (k_out is None):
        raise ValueError("gqa_rope needs positions, and k and k_out together")
    _on_device(k=k, k_out=k_out)
    rope = Rope(inv_freq, positions, interleaved, attn_factor, q, out, inverse)
    rows, _, d = q.shape
    a = rope._args(int(rows), q.dtype, int(d))
    ks = kos = hkv = 0
    if k is not None:
        ks, kos, hkv = _rows("k", k), _rows("k_out", k_out, k), int(k.shape[1])
        if k.shape[0] != rows or k.shape[2] != d or k.dtype != q.dtype:
            raise ValueError("k must have q's rows, head dim and type")
    return PreparedOp(load().gqa_rope,
                      (ctypes.byref(a), _ptr(k), ks, _ptr(k_out), kos, int(rows), hkv, int(d),
                       _dtype_code(q), _stream_handle(stream)), "gqa_rope", (rope, a, k, k_out))


def gqa_rope(q, positions, inv_freq, out, k=None, k_out=None, interleaved=False, attn_factor=1.0,
             inverse=False, stream=None):
    """Rotate query rows (and key rows) by their positions into ``out`` (and
    ``k_out``); ``inverse`` rotates back, which is the gradient.  Rows may be
    slices of a packed projection.  See gqa_prefill.h; returns ``out``."""
    _marshal_rope(q, positions, inv_freq, out, k, k_out, interleaved, attn_factor, inverse,
                  stream)()
    return out


def _marshal_cache_write(k, v, cu_seqlens_q, prefix_lens, kv_page_indptr, kv_page_indices, k_pages,
                         v_pages, k_scales=None, v_scales=None, rope=None, stream=None):
    _on_device(k=k, v=v, cu_seqlens_q=cu_seqlens_q, prefix_lens=prefix_lens,
               kv_page_indptr=kv_page_indptr, kv_page_indices=kv_page_indices, k_pages=k_pages,
               v_pages=v_pages, k_scales=k_scales, v_scales=v_scales)
    _int32(cu_seqlens_q=cu_seqlens_q, prefix_lens=prefix_lens, kv_page_indptr=kv_page_indptr,
           kv_page_indices=kv_page_indices)
    ks, vs = _rows("k", k), _rows("v", v)
    if k.shape != v.shape or k.dtype != v.dtype:
        raise ValueError("k and v must agree in shape and type")
    n = _lengths(cu_seqlens_q, prefix_lens, kv_page_indptr)
    kind, pages, page_size, hkv, d = _pool(k_pages, v_pages, k_scales, v_scales, k.dtype)
    rows = int(k.shape[0])
    if (int(k.shape[1]), int(k.shape[2])) != (hkv, d):
        raise ValueError("k must have the pages' heads and head dim")
    a = rope._args(rows, k.dtype, d) if rope is not None else None
    return PreparedOp(load().gqa_cache_write,
                      (_ptr(k), ks, _ptr(v), vs, _ptr(cu_seqlens_q), _ptr(prefix_lens),
                       _ptr(kv_page_indptr), _ptr(kv_page_indices), int(kv_page_indices.numel()),
                       page_size, pages, n, rows, hkv, d, _dtype_code(k), kind, _ptr(k_pages),
                       _ptr(v_pages), _ptr(k_scales), _ptr(v_scales),
                       None if a is None else ctypes.byref(a), _stream_handle(stream)),
                      "gqa_cache_write", (rope, a, k, v, cu_seqlens_q, prefix_lens, kv_page_indptr,
                                          kv_page_indices, k_pages, v_pages, k_scales, v_scales))


def gqa_cache_write(k, v, cu_seqlens_q, prefix_lens, kv_page_indptr, kv_page_indices, k_pages,
                    v_pages, k_scales=None, v_scales=None, rope=None, stream=None):
    """Write the new tokens' K and V into their pages (16-bit, or e4m3 with
    byte scales), rotating k, and rope.q, on the way.  See gqa_prefill.h."""
    _marshal_cache_write(k, v, cu_seqlens_q, prefix_lens, kv_page_indptr, kv_page_indices, k_pages,
                         v_pages, k_scales, v_scales, rope, stream)()


def _marshal_cache_read(k_pages, v_pages, kv_page_indptr, kv_page_indices, kv_indptr, k_out, v_out,
                        first_keys=None, k_scales=None, v_scales=None, stream=None):
    _on_device(k_pages=k_pages, v_pages=v_pages, kv_page_indptr=kv_page_indptr,
               kv_page_indices=kv_page_indices, kv_indptr=kv_indptr, k_out=k_out, v_out=v_out,
               first_keys=first_keys, k_scales=k_scales, v_scales=v_scales)
    _int32(kv_page_indptr=kv_page_indptr, kv_page_indices=kv_page_indices, kv_indptr=kv_indptr,
           first_keys=first_keys)
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t.dim() != 3 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [rows, heads, d] tensor")
    if k_out.shape != v_out.shape or k_out.dtype != v_out.dtype:
        raise ValueError("k_out and v_out must agree in shape and type")
    kind, pages, page_size, hkv, d = _pool(k_pages, v_pages, k_scales, v_scales, k_out.dtype)
    if (int(k_out.shape[1]), int(k_out.shape[2])) != (hkv, d):
        raise ValueError("k_out must have the pages' heads and head dim")
    n = int(kv_page_indptr.numel()) - 1
    if kv_indptr.numel() != n + 1 or (first_keys is not None and first_keys.numel() != n):
        raise ValueError("kv_indptr and first_keys must match kv_page_indptr")
    return PreparedOp(load().gqa_cache_read,
                      (_ptr(k_pages), _ptr(v_pages), _ptr(k_scales), _ptr(v_scales), kind,
                       _ptr(kv_page_indptr), _ptr(kv_page_indices), int(kv_page_indices.numel()),
                       page_size, pages, _ptr(kv_indptr), _ptr(first_keys), n,
                       int(k_out.shape[0]), hkv, d, _dtype_code(k_out), _ptr(k_out), _ptr(v_out),
                       _stream_handle(stream)), "gqa_cache_read",
                      (k_pages, v_pages, k_scales, v_scales, kv_page_indptr, kv_page_indices,
                       kv_indptr, first_keys, k_out, v_out))


def gqa_cache_read(k_pages, v_pages, kv_page_indptr, kv_page_indices, kv_indptr, k_out, v_out,
                   first_keys=None, k_scales=None, v_scales=None, stream=None):
    """Gather keys and values out of the pages into contiguous 16-bit rows
    (see gqa_prefill.h).  Returns (k_out, v_out)."""
    _marshal_cache_read(k_pages, v_pages, kv_page_indptr, kv_page_indices, kv_indptr, k_out, v_out,
                        first_keys, k_scales, v_scales, stream)()
    return k_out, v_out


def _cache_code(cache) -> int:
    if isinstance(cache, int):
        return cache
    if str(cache) not in ("16", "e4m3"):
        raise ValueError('cache must be "16" or "e4m3"')
    return GQA_CACHE_E4M3 if str(cache) == "e4m3" else GQA_CACHE_16


def cache_attention_workspace(num_seqs, total_q, max_seqlen_q, hq, hkv, d, dtype, cache="16"):
    """Workspace bytes of a gqa_cache_attention call with these shapes;
    ``cache`` is "16" or "e4m3" (or GQA_CACHE_*)."""
    nbytes = ctypes.c_size_t(0)
    code = dtype if isinstance(dtype, int) else (
        GQA_BF16 if "bf16" in str(dtype) or "bfloat16" in str(dtype) else GQA_F16)
    rc = load().gqa_cache_attention_workspace(int(num_seqs), int(total_q), int(max_seqlen_q),
                                              int(hq), int(hkv), int(d), code, _cache_code(cache),
                                              ctypes.byref(nbytes))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_cache_attention_workspace")
    return nbytes.value


def _marshal_cache_attention(q, k_pages, v_pages, cu_seqlens_q, prefix_lens, kv_page_indptr,
                             kv_page_indices, scale, workspace, window=0, sinks=None,
                             smooth_softmax=False, k_scales=None, v_scales=None, custom_mask=None,
                             mask_indptr=None, depths=None, out=None, lse=None, stream=None,
                             max_seqlen_q=0):
    import torch
    _on_device(q=q, k_pages=k_pages, v_pages=v_pages, cu_seqlens_q=cu_seqlens_q,
               prefix_lens=prefix_lens, kv_page_indptr=kv_page_indptr,
               kv_page_indices=kv_page_indices, workspace=workspace, sinks=sinks,
               k_scales=k_scales, v_scales=v_scales, custom_mask=custom_mask,
               mask_indptr=mask_indptr, depths=depths, out=out, lse=lse)
    if out is None:
        raise ValueError("out is required")
    for name, t in (("q", q), ("out", out)):
        if t.dim() != 3 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [rows, heads, d] tensor")
    _int32(cu_seqlens_q=cu_seqlens_q, prefix_lens=prefix_lens, kv_page_indptr=kv_page_indptr,
           kv_page_indices=kv_page_indices, mask_indptr=mask_indptr, depths=depths)
    total_q, hq, d = (int(n) for n in q.shape)
    kind, pages, page_size, hkv, pd = _pool(k_pages, v_pages, k_scales, v_scales, q.dtype)
    n = _lengths(cu_seqlens_q, prefix_lens, kv_page_indptr)
    if pd != d or out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("q, out and the pages must agree in head dim and type")
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (total_q, hq)
                            or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [rows, heads] tensor")
    if sinks is not None and (sinks.dtype != torch.float32 or sinks.numel() != hq
                              or not sinks.is_contiguous()):
        raise ValueError("sinks must be a contiguous float32 tensor of one value per head")
    if (custom_mask is None) != (mask_indptr is None):
        raise ValueError("custom_mask and mask_indptr go together")
    if custom_mask is not None and (custom_mask.element_size() != 4
                                    or not custom_mask.is_contiguous()
                                    or mask_indptr.numel() != n + 1):
        raise ValueError("custom_mask must be contiguous 32-bit words, one mask_indptr entry more "
                         "than sequences")
    if depths is not None and depths.numel() != total_q:
        raise ValueError("depths must have one entry per row")
    words = 0 if custom_mask is None else int(custom_mask.numel())
    if words == 0 and custom_mask is not None:
        custom_mask = mask_indptr  # no words, hence no tokens: any address will do
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return PreparedOp(load().gqa_cache_attention,
                      (_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scales), _ptr(v_scales), kind,
                       _ptr(cu_seqlens_q), _ptr(prefix_lens), _ptr(kv_page_indptr),
                       _ptr(kv_page_indices), int(kv_page_indices.numel()), page_size, pages, n,
                       total_q, int(max_seqlen_q), hq, hkv, d, _dtype_code(q), float(scale),
                       int(window), _ptr(sinks), 1 if smooth_softmax else 0, _ptr(custom_mask),
                       _ptr(mask_indptr), words, _ptr(depths), _ptr(out), _ptr(lse),
                       _ptr(workspace), nbytes, _stream_handle(stream)), "gqa_cache_attention",
                      (q, k_pages, v_pages, k_scales, v_scales, cu_seqlens_q, prefix_lens,
                       kv_page_indptr, kv_page_indices, sinks, custom_mask, mask_indptr, depths,
                       out, lse, workspace))


def gqa_cache_attention(q, k_pages, v_pages, cu_seqlens_q, prefix_lens, kv_page_indptr,
                        kv_page_indices, scale, workspace, window=0, sinks=None,
                        smooth_softmax=False, k_scales=None, v_scales=None, custom_mask=None,
                        mask_indptr=None, depths=None, out=None, lse=None, stream=None,
                        max_seqlen_q=0):
    """Attention of a few new tokens per sequence (a decoded token, or a tree
    of drafted ones) over a paged 16-bit or e4m3 cache (see gqa_prefill.h);
    ``workspace`` is a device tensor of at least
    ``cache_attention_workspace(...)`` bytes.  Returns ``out``."""
    _marshal_cache_attention(q, k_pages, v_pages, cu_seqlens_q, prefix_lens, kv_page_indptr,
                             kv_page_indices, scale, workspace, window, sinks, smooth_softmax,
                             k_scales, v_scales, custom_mask, mask_indptr, depths, out, lse, stream,
                             max_seqlen_q)()
    return out


# ------------------------------------------------------------------ gradients
def _type_code(dtype) -> int:
    if isinstance(dtype, int):
        return dtype
    codes = {"bf16": GQA_BF16, "bfloat16": GQA_BF16, "f16": GQA_F16, "float16": GQA_F16}
    name = str(dtype).replace("torch.", "")
    if name not in codes:
        raise TypeError(f"dtype must be float16 or bfloat16, got {dtype}")
    return codes[name]


def prefill_backward_workspace(num_seqs, total_q, total_kv, hq, hkv, d, dtype):
    """Workspace bytes of a gqa_prefill_backward call with these shapes."""
    nbytes = ctypes.c_size_t(0)
    rc = load().gqa_prefill_backward_workspace(int(num_seqs), int(total_q), int(total_kv), int(hq),
                                               int(hkv), int(d), _type_code(dtype),
                                               ctypes.byref(nbytes))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_prefill_backward_workspace")
    return nbytes.value


def _float32(shape, **tensors):
    import torch
    for name, t in tensors.items():
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shape
                              or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 tensor {list(shape)}")


def _marshal_prefill_backward(q, k, v, cu_seqlens_q, prefix_lens, kv_indptr, scale, out, lse, dout,
                              dq, dk, dv, workspace, window=0, sinks=None, dsinks=None, dlse=None,
                              stream=None):
    _on_device(q=q, k=k, v=v, cu_seqlens_q=cu_seqlens_q, prefix_lens=prefix_lens,
               kv_indptr=kv_indptr, out=out, lse=lse, dout=dout, dq=dq, dk=dk, dv=dv,
               workspace=workspace, sinks=sinks, dsinks=dsinks, dlse=dlse)
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out), ("dout", dout), ("dq", dq),
                    ("dk", dk), ("dv", dv)):
        if t.dim() != 3 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [rows, heads, d] tensor")
    for name, t, like in (("out", out, q), ("dout", dout, q), ("dq", dq, q), ("v", v, k),
                          ("dk", dk, k), ("dv", dv, k)):
        if t.shape != like.shape or t.dtype != q.dtype:
            raise ValueError(f"{name} must have the shape and type of its input")
    if k.dtype != q.dtype or k.shape[2] != q.shape[2]:
        raise ValueError("k must have q's head dim and type")
    _int32(cu_seqlens_q=cu_seqlens_q, prefix_lens=prefix_lens, kv_indptr=kv_indptr)
    n = int(prefix_lens.numel())
    if cu_seqlens_q.numel() != n + 1 or kv_indptr.numel() != n + 1:
        raise ValueError("cu_seqlens_q and kv_indptr must have one entry more than prefix_lens")
    total_q, hq, d = (int(x) for x in q.shape)
    total_kv, hkv = int(k.shape[0]), int(k.shape[1])
    if lse is None:
        raise ValueError("lse is required")
    _float32((total_q, hq), lse=lse, dlse=dlse)
    _float32((hq,), sinks=sinks, dsinks=dsinks)
    if dsinks is not None and sinks is None:
        raise ValueError("dsinks needs sinks")
    if dsinks is None:
        sinks = None  # their gradient is left out; lse holds their weight
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return PreparedOp(load().gqa_prefill_backward,
                      (_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens_q), _ptr(prefix_lens),
                       _ptr(kv_indptr), n, total_q, total_kv, hq, hkv, d, _dtype_code(q),
                       float(scale), int(window), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dlse),
                       _ptr(sinks), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dsinks), _ptr(workspace),
                       nbytes, _stream_handle(stream)), "gqa_prefill_backward",
                      (q, k, v, cu_seqlens_q, prefix_lens, kv_indptr, out, lse, dout, dlse, sinks,
                       dq, dk, dv, dsinks, workspace))


def gqa_prefill_backward(q, k, v, cu_seqlens_q, prefix_lens, kv_indptr, scale, out, lse, dout, dq,
                         dk, dv, workspace, window=0, sinks=None, dsinks=None, dlse=None,
                         stream=None):
    """The gradient of gqa_flash_prefill (see gqa_prefill.h) into ``dq``,
    ``dk``, ``dv`` and, when given, ``dsinks``; ``workspace`` is a device
    tensor of at least ``prefill_backward_workspace(...)`` bytes.  Returns
    (dq, dk, dv)."""
    _marshal_prefill_backward(q, k, v, cu_seqlens_q, prefix_lens, kv_indptr, scale, out, lse, dout,
                              dq, dk, dv, workspace, window, sinks, dsinks, dlse, stream)()
    return dq, dk, dv


def prefill_backward(batch, out, lse, dout, dlse=None, workspace=None, stream=None):
    """gqa_prefill_backward of one ``workloads.Batch`` already on the GPU, from
    what ``prefill`` returned and the gradient of its out; allocates the
    results (and the workspace, when not given) with torch.  Returns
    (dq, dk, dv, dsinks), dsinks None for a batch without sinks."""
    import torch
    dq, dk, dv = (_result(t.shape, t.dtype, t.device, stream) for t in (batch.q, batch.k, batch.v))
    dsinks = None
    if batch.sinks is not None:
        dsinks = _result(batch.sinks.shape, torch.float32, batch.q.device, stream)
    if workspace is None:
        size = prefill_backward_workspace(batch.num_seqs, batch.total_q, batch.total_kv, batch.hq,
                                          batch.hkv, batch.d, batch.dtype_name)
        with _allocating(stream):
            workspace = torch.empty(size, dtype=torch.uint8, device=batch.q.device)
    gqa_prefill_backward(batch.q, batch.k, batch.v, batch.cu_seqlens_q, batch.prefix_lens,
                         batch.kv_indptr, batch.scale, out, lse, dout, dq, dk, dv, workspace,
                         window=batch.window, sinks=batch.sinks, dsinks=dsinks, dlse=dlse,
                         stream=stream)
    return dq, dk, dv, dsinks


# ------------------------------------------------------------------ the norm
def _norm_rows(name, t, like=None):
    """(rows, heads, n, row stride) of [rows, n] or [rows, heads, n] with
    packed heads."""
    if t.dim() == 2:
        t = t.unsqueeze(1)
    if like is not None and tuple(t.shape) != like:
        raise ValueError(f"{name} must have the shape of the rows")
    stride = _rows(name, t)
    return (*(int(x) for x in t.shape), stride)


def _norm_type(name, t, dtype) -> int:
    """GQA_* code of a residual stream or a weight: the rows' type, or float32."""
    import torch
    if t.dtype == torch.float32:
        return GQA_F32
    if t.dtype != dtype:
        raise TypeError(f"{name} must have the rows' type or be float32, got {t.dtype}")
    return _dtype_code(t)


def _norm_weight(weight, n, dtype) -> int:
    if weight.dim() != 1 or weight.numel() != n or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous vector of one value per column")
    return _norm_type("weight", weight, dtype)


def _norm_stream(name, t, shape):
    if t is not None and (tuple(t.unsqueeze(1).shape if t.dim() == 2 else t.shape) != shape
                          or not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous and have the shape of the rows")


def _norm_rstd(rstd, rows, heads):
    import torch
    if rstd is not None and (rstd.dtype != torch.float32 or rstd.numel() != rows * heads
                             or not rstd.is_contiguous()):
        raise ValueError("rstd must be a contiguous float32 tensor of one value per row and head")


def _marshal_rms_norm(x, weight, out, eps=1e-5, offset=0.0, residual=None, residual_out=None,
                      scales=None, rstd=None, stream=None):
    import torch
    _on_device(x=x, weight=weight, out=out, residual=residual, residual_out=residual_out,
               scales=scales, rstd=rstd)
    rows, heads, n, xs = _norm_rows("x", x)
    shape = (rows, heads, n)
    os_ = _norm_rows("out", out, shape)[3]
    code, wtype = _dtype_code(x), _norm_weight(weight, n, x.dtype)
    if (residual is None) != (residual_out is None):
        raise ValueError("residual and residual_out go together")
    _norm_stream("residual", residual, shape)
    _norm_stream("residual_out", residual_out, shape)
    stype = code
    if residual is not None:
        stype = _norm_type("residual", residual, x.dtype)
        if residual_out.dtype != residual.dtype:
            raise ValueError("residual_out must have residual's type")
    _norm_rstd(rstd, rows, heads)
    kind, group = GQA_CACHE_16, 0
    if scales is not None:
        if out.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise TypeError(f"out with scales must be e4m3, got {out.dtype}")
        groups = int(scales.shape[-1]) if scales.dim() == out.dim() else 0
        if (groups <= 0 or n % groups != 0 or scales.element_size() != 1
                or scales.shape[:-1] != out.shape[:-1] or not scales.is_contiguous()):
            raise ValueError("scales must be a contiguous byte tensor [rows, heads, groups], as many "
                             "dimensions as out, whose groups divide the columns")
        kind, group = GQA_CACHE_E4M3, n // groups
    elif out.dtype != x.dtype:
        raise TypeError(f"out must have x's type, or be e4m3 with scales, got {out.dtype}")
    return PreparedOp(load().gqa_rms_norm,
                      (_ptr(x), xs, _ptr(residual), _ptr(residual_out), stype, _ptr(weight), wtype,
                       float(offset), float(eps), rows, heads, n, code, kind, group, _ptr(out), os_,
                       _ptr(scales), _ptr(rstd), _stream_handle(stream)), "gqa_rms_norm",
                      (x, residual, residual_out, weight, out, scales, rstd))


def gqa_rms_norm(x, weight, out, eps=1e-5, offset=0.0, residual=None, residual_out=None,
                 scales=None, rstd=None, stream=None):
    """Root-mean-square norm of each row's last dimension, x [rows, n] or
    [rows, heads, n] (a slice of a packed projection will do), after the
    addition of ``residual`` (into ``residual_out``), into ``out``: x's type, or
    e4m3 with byte ``scales`` [.., n / group].  ``rstd`` is kept for the
    gradient.  See gqa_prefill.h; returns ``out``."""
    _marshal_rms_norm(x, weight, out, eps, offset, residual, residual_out, scales, rstd, stream)()
    return out


def rms_norm(x, weight, eps=1e-5, offset=0.0, residual=None, group=None, with_rstd=False,
             stream=None):
    """gqa_rms_norm into new tensors; ``group`` values share a scale of an e4m3
    output (None: an output of x's type).  Returns (out, scales or None, h, rstd
    or None) with h the sum with the residual, or x itself."""
    import torch
    dtype = x.dtype if group is None else torch.float8_e4m3fn
    out = _result(x.shape, dtype, x.device, stream)
    scales = h = rstd = None
    if group is not None:
        if group <= 0 or x.shape[-1] % group != 0:
            raise ValueError("group must divide the columns")
        scales = _result((*x.shape[:-1], x.shape[-1] // group), torch.uint8, x.device, stream)
    if residual is not None:
        h = _result(x.shape, residual.dtype, x.device, stream)
    if with_rstd:
        rstd = _result(x.shape[:-1], torch.float32, x.device, stream)
    gqa_rms_norm(x, weight, out, eps, offset, residual, h, scales, rstd, stream)
    return out, scales, x if h is None else h, rstd


def rms_norm_backward_workspace(rows, heads, n, dtype):
    """Workspace bytes of a gqa_rms_norm_backward call with these shapes."""
    nbytes = ctypes.c_size_t(0)
    rc = load().gqa_rms_norm_backward_workspace(int(rows), int(heads), int(n), _type_code(dtype),
                                                ctypes.byref(nbytes))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_rms_norm_backward_workspace")
    return nbytes.value


def _marshal_rms_norm_backward(dy, h, weight, rstd, dx=None, dresidual=None, dweight=None,
                               workspace=None, offset=0.0, dh=None, stream=None):
    import torch
    _on_device(dy=dy, h=h, weight=weight, rstd=rstd, dx=dx, dresidual=dresidual, dweight=dweight,
               workspace=workspace, dh=dh)
    if rstd is None:
        raise ValueError("rstd is required")
    rows, heads, n, ys = _norm_rows("dy", dy)
    shape = (rows, heads, n)
    hs = _norm_rows("h", h, shape)[3]
    code, wtype = _dtype_code(dy), _norm_weight(weight, n, dy.dtype)
    stype = _norm_type("h", h, dy.dtype)
    xs = heads * n
    if dx is not None:
        xs = _norm_rows("dx", dx, shape)[3]
        if dx.dtype != dy.dtype:
            raise ValueError("dx must have dy's type")
    for name, t in (("dh", dh), ("dresidual", dresidual)):
        _norm_stream(name, t, shape)
        if t is not None and t.dtype != h.dtype:
            raise ValueError(f"{name} must have h's type")
    _norm_rstd(rstd, rows, heads)
    _float32((n,), dweight=dweight)
    if dweight is not None and workspace is None and rows > 0:
        raise ValueError("dweight needs a workspace")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return PreparedOp(load().gqa_rms_norm_backward,
                      (_ptr(dy), ys, _ptr(h), hs, stype, _ptr(rstd), _ptr(weight), wtype,
                       float(offset), _ptr(dh), rows, heads, n, code, _ptr(dx), xs,
                       _ptr(dresidual), _ptr(dweight), _ptr(workspace), nbytes,
                       _stream_handle(stream)), "gqa_rms_norm_backward",
                      (dy, h, rstd, weight, dh, dx, dresidual, dweight, workspace))


def gqa_rms_norm_backward(dy, h, weight, rstd, dx=None, dresidual=None, dweight=None,
                          workspace=None, offset=0.0, dh=None, stream=None):
    """The gradient of gqa_rms_norm (see gqa_prefill.h) into those of ``dx``,
    ``dresidual`` and ``dweight`` that are given, from ``dy`` and ``dh``, the
    gradient that reaches h another way; ``dweight`` needs a workspace of
    ``rms_norm_backward_workspace(...)`` bytes.  Returns ``dx``."""
    _marshal_rms_norm_backward(dy, h, weight, rstd, dx, dresidual, dweight, workspace, offset, dh,
                               stream)()
    return dx


def rms_norm_backward(dy, h, weight, rstd, offset=0.0, dh=None, workspace=None, stream=None):
    """gqa_rms_norm_backward into new tensors.  Returns (dx, dresidual,
    dweight): dx in dy's type; dresidual is dx itself unless the stream h is
    wider."""
    import torch
    rows, heads, n = (*dy.shape[:1], 1, *dy.shape[1:]) if dy.dim() == 2 else dy.shape
    dx = _result(dy.shape, dy.dtype, dy.device, stream)
    dresidual = None if h.dtype == dy.dtype else _result(h.shape, h.dtype, h.device, stream)
    dweight = _result((n,), torch.float32, dy.device, stream)
    if workspace is None:
        with _allocating(stream):
            workspace = torch.empty(rms_norm_backward_workspace(rows, heads, n, dy.dtype),
                                    dtype=torch.uint8, device=dy.device)
    gqa_rms_norm_backward(dy, h, weight, rstd, dx, dresidual, dweight, workspace, offset, dh, stream)
    return dx, dx if dresidual is None else dresidual, dweight


_MARSHAL = {gqa_rope: _marshal_rope, gqa_cache_write: _marshal_cache_write,
            gqa_cache_read: _marshal_cache_read, gqa_cache_attention: _marshal_cache_attention,
            gqa_prefill_backward: _marshal_prefill_backward, gqa_rms_norm: _marshal_rms_norm,
            gqa_rms_norm_backward: _marshal_rms_norm_backward}


def cache_write(batch, cache, rope=None, stream=None):
    """gqa_cache_write of the new tokens of one ``workloads.Batch`` (its q, k
    and v hold the new tokens' rows) into a ``workloads.Cache``, both on the
    GPU."""
    gqa_cache_write(batch.k, batch.v, batch.cu_seqlens_q, batch.prefix_lens, cache.page_indptr,
                    cache.page_indices, cache.k_pages, cache.v_pages, k_scales=cache.k_scales,
                    v_scales=cache.v_scales, rope=rope, stream=stream)


def cache_read(cache, kv_indptr, total_kv, dtype, first_keys=None, stream=None):
    """gqa_cache_read of a ``workloads.Cache`` into new rows.  Returns (k, v)."""
    _, _, hkv, d = cache.k_pages.shape
    k, v = (_result((total_kv, hkv, d), dtype, cache.k_pages.device, stream) for _ in range(2))
    return gqa_cache_read(cache.k_pages, cache.v_pages, cache.page_indptr, cache.page_indices,
                          kv_indptr, k, v, first_keys=first_keys, k_scales=cache.k_scales,
                          v_scales=cache.v_scales, stream=stream)


def cache_attention(batch, cache, q=None, custom_mask=None, mask_indptr=None, depths=None,
                    workspace=None, out=None, lse=None, with_lse=True, stream=None):
    """gqa_cache_attention of one ``workloads.Batch``'s queries (or ``q`` in
    their place, the rotated ones) over a ``workloads.Cache``; allocates
    workspace, out and lse with torch when not given.  Returns (out, lse)."""
    import torch
    q = batch.q if q is None else q
    out, lse = _outputs(q, out, lse, with_lse, stream)
    if workspace is None:
        size = cache_attention_workspace(batch.num_seqs, batch.total_q, batch.max_seqlen_q,
                                         batch.hq, batch.hkv, batch.d, batch.dtype_name, cache.kind)
        with _allocating(stream):
            workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
    gqa_cache_attention(q, cache.k_pages, cache.v_pages, batch.cu_seqlens_q, batch.prefix_lens,
                        cache.page_indptr, cache.page_indices, batch.scale, workspace,
                        window=batch.window, sinks=batch.sinks, smooth_softmax=batch.smooth,
                        k_scales=cache.k_scales, v_scales=cache.v_scales, custom_mask=custom_mask,
                        mask_indptr=mask_indptr, depths=depths, out=out, lse=lse, stream=stream,
                        max_seqlen_q=batch.max_seqlen_q)
    return out, lse


def set_call_flags(flags: int) -> None:
    """Flags for the calling thread's later calls (gqa_prefill_set_call_flags):
    FLAG_METADATA_READY, or 0."""
    rc = load().gqa_prefill_set_call_flags(int(flags))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_prefill_set_call_flags")


def get_call_flags() -> int:
    return int(load().gqa_prefill_get_call_flags())


def plan(num_seqs, total_q, max_seqlen_q, hq, hkv, d, dtype, window) -> dict:
    """Host-only launch plan (rows_per_unit, block_n, kv_stages, ctas_per_sm,
    grid, max_units, q_tiles) for a call with these shapes."""
    p = _Plan()
    code = dtype if isinstance(dtype, int) else (GQA_BF16 if "bf16" in str(dtype) else GQA_F16)
    rc = load().gqa_prefill_plan(int(num_seqs), int(total_q), int(max_seqlen_q), int(hq),
                                 int(hkv), int(d), code, int(window), ctypes.byref(p))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_prefill_plan")
    return {f: getattr(p, f) for f, _ in _Plan._fields_}


def force_block_n(block_n: int) -> None:
    rc = load().gqa_prefill_force_block_n(int(block_n))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_prefill_force_block_n")


def force_q_tiles(q_tiles: int) -> None:
    """Pin 1 or 2 query tiles per work unit for later calls (0: the cache's choice)."""
    rc = load().gqa_prefill_force_q_tiles(int(q_tiles))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_prefill_force_q_tiles")


def set_tuning(enable: bool) -> None:
    """Turn the configuration cache's timed sweep on or off (see gqa_prefill.h)."""
    rc = load().gqa_prefill_set_tuning(1 if enable else 0)
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_prefill_set_tuning")


def clear_config_cache() -> None:
    load().gqa_prefill_clear_config_cache()


def config_block_n(total_q, max_seqlen_q, hq, hkv, d, dtype, window):
    """(block_n, q_tiles, tuned) cached for these shapes; block_n 0 = no entry
    yet."""
    bn, qt, tuned = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    code = dtype if isinstance(dtype, int) else (GQA_BF16 if "bf16" in str(dtype) else GQA_F16)
    rc = load().gqa_prefill_config_block_n(int(total_q), int(max_seqlen_q), int(hq), int(hkv),
                                           int(d), code, int(window), ctypes.byref(bn),
                                           ctypes.byref(qt), ctypes.byref(tuned))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_prefill_config_block_n")
    return bn.value, qt.value, bool(tuned.value)


def selftest_timeout(timeout_ms: int = 50, stream=None) -> int:
    """Run the bounded-wait self-test; returns the device status word it read."""
    st = ctypes.c_int(0)
    rc = load().gqa_prefill_selftest_timeout(int(timeout_ms), _stream_handle(stream),
                                             ctypes.byref(st))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_prefill_selftest_timeout")
    return st.value


def get_stream_status(stream=None) -> int:
    """Read and clear the device status word in the order of ``stream``
    (default: the current stream), waiting for that stream only."""
    v = ctypes.c_int(0)
    rc = load().gqa_prefill_get_stream_status(_stream_handle(stream), ctypes.byref(v))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_prefill_get_stream_status")
    return v.value


def get_device_status() -> int:
    """Read and clear the device status word (synchronises the device)."""
    v = ctypes.c_int(0)
    rc = load().gqa_prefill_get_device_status(ctypes.byref(v))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_prefill_get_device_status")
    return v.value
