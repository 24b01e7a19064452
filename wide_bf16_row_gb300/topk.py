"""Python binding over ``libtf_topk.so`` (C ABI in ``include/tf_topk.h``).

Argument marshalling only: every step runs in the library's CUDA kernels.
PyTorch supplies device memory and the current stream.  If the library has
not been built, every entry point raises -- there is no fallback.

Tensor-level calls: ``topk_bf16`` (bf16 rows, k <= 64, any launch plan),
``select_topk`` (bf16 / fp16 / fp32 rows, k <= 1024), ``merge_bf16``
(per-shard lists into each row's top k), ``nucleus_bf16`` (top-p
probabilities over the lists), ``head_topk_bf16`` (the draft head's
product and the top-k in one kernel), ``head_loss_bf16`` and
``head_loss_grad_bf16`` (the head's cross entropy and its gradient without the
logits), ``route_experts`` and ``route_experts_grad`` (each token's experts and
their weights), ``sort_by_expert``, ``gather_tokens``, ``combine_tokens`` and
their gradients (tokens sorted by expert and back), ``quantize_tokens_fp8`` and
``product_fp8`` (rows in 8 bits and their products with weights in 8 bits),
``penalize_logits`` (penalties, biases and masks before the top-k).  The raw C entry points are exposed under their C names.
"""
from __future__ import annotations

import ctypes
from pathlib import Path
from typing import Any, NamedTuple

PKG = Path(__file__).resolve().parent
LIBRARY = PKG / "libtf_topk.so"

# status codes (include/tf_topk.h)
OK, ERR_NULL, ERR_SHAPE, ERR_K, ERR_ALIGN, ERR_PLAN, ERR_DEVICE, ERR_CUDA = range(8)
ERR_SCRATCH = 8  # tf_topk_bf16_noalloc only
ERR_ARG = 9  # tf_topk_nucleus_bf16 only
ERR_DTYPE = 10  # tf_topk_select only
DTYPE_BF16, DTYPE_F16, DTYPE_F32 = 0, 1, 2
PLAN_WIDE = 64  # tf_topk_select_with_plan: the wide kernel

# launch plans (include/tf_topk.h)
PLAN_AUTO, PLAN_SINGLE, PLAN_STREAM = 0, 1, 32
PLAN_CLUSTER = {2: 2, 4: 4, 8: 8, 16: 16}
PLANS = (PLAN_AUTO, PLAN_SINGLE, 2, 4, 8, 16, PLAN_STREAM)

_lib = None


class TopkError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"tf_topk status {status}: {message}")
        self.status = status


def library() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it was never built."""
    global _lib
    if _lib is None:
        if not LIBRARY.exists():
            raise ImportError(f"{LIBRARY} is missing: build it with "
                              "`python -m wide_bf16_row_gb300.build` (no CPU fallback exists)")
        lib = ctypes.CDLL(str(LIBRARY))
        c_i64, c_i32, c_p = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
        lib.tf_topk_bf16.restype = ctypes.c_int
        lib.tf_topk_bf16.argtypes = [c_p, c_i64, c_i64, c_i64, c_i32, c_p, c_p, c_p, c_p, c_p]
        lib.tf_topk_bf16_with_plan.restype = ctypes.c_int
        lib.tf_topk_bf16_with_plan.argtypes = [c_p, c_i64, c_i64, c_i64, c_i32, c_p, c_p, c_p,
                                               c_p, c_i32, c_p]
        lib.tf_topk_merge_bf16.restype = ctypes.c_int
        lib.tf_topk_merge_bf16.argtypes = [c_p, c_p, c_p, c_p, c_i64, c_i32, c_i32, c_p, c_i32, c_p, c_p, c_p,
                                           c_p, c_p]
        lib.tf_topk_bf16_noalloc.restype = ctypes.c_int
        lib.tf_topk_bf16_noalloc.argtypes = [c_p, c_i64, c_i64, c_i64, c_i32, c_p, c_p, c_p, c_p, c_p]
        lib.tf_topk_nucleus_bf16.restype = ctypes.c_int
        lib.tf_topk_nucleus_bf16.argtypes = [c_p, c_p, c_i64, c_i32, ctypes.c_float, ctypes.c_float, c_p, c_p, c_p]
        lib.tf_topk_nucleus.restype = ctypes.c_int
        lib.tf_topk_nucleus.argtypes = [c_p, c_i32, c_p, c_i64, c_i32, ctypes.c_float, ctypes.c_float, c_p, c_p, c_p]
        lib.tf_topk_select.restype = ctypes.c_int
        lib.tf_topk_select.argtypes = [c_p, c_i32, c_i64, c_i64, c_i64, c_i32, c_p, c_p, c_p, c_p, c_p]
        lib.tf_topk_select_with_plan.restype = ctypes.c_int
        lib.tf_topk_select_with_plan.argtypes = [c_p, c_i32, c_i64, c_i64, c_i64, c_i32, c_p, c_p, c_p, c_p,
                                                 c_i32, c_p]
        lib.tf_topk_select_max_k.restype = c_i32
        lib.tf_topk_select_max_k.argtypes = []
        lib.tf_topk_device_fault.restype = ctypes.c_int
        lib.tf_topk_device_fault.argtypes = []
        lib.tf_topk_bf16_plan.restype = c_i32
        lib.tf_topk_bf16_plan.argtypes = [c_i64, c_i64, c_i32]
        for name in ("tf_topk_bf16_max_k", "tf_topk_bf16_max_spans", "tf_topk_bf16_cta_threads",
                     "tf_topk_bf16_chunk_columns"):
            getattr(lib, name).restype = c_i32
            getattr(lib, name).argtypes = []
        lib.tf_topk_head_bf16.restype = ctypes.c_int
        lib.tf_topk_head_bf16.argtypes = [c_p, c_p, c_i32, c_i32, c_i64, c_i32, c_p, ctypes.c_size_t, c_p, c_p,
                                          c_p, c_p, c_p]
        lib.tf_topk_head_bf16_workspace.restype = ctypes.c_size_t
        lib.tf_topk_head_bf16_workspace.argtypes = [c_i32, c_i32]
        c_size = ctypes.c_size_t
        lib.tf_topk_head_loss_bf16.restype = ctypes.c_int
        lib.tf_topk_head_loss_bf16.argtypes = [c_p, c_i64, c_p, c_i64, c_i64, c_i32, c_i64, c_p, c_i32, c_i64, c_p,
                                               c_size, c_p, c_p, c_p]
        lib.tf_topk_head_loss_bf16_workspace.restype = c_size
        lib.tf_topk_head_loss_bf16_workspace.argtypes = [c_i64, c_i32, c_i64]
        lib.tf_topk_head_loss_grad_bf16.restype = ctypes.c_int
        lib.tf_topk_head_loss_grad_bf16.argtypes = [c_p, c_i64, c_p, c_i64, c_i64, c_i32, c_i64, c_p, c_i32, c_i64,
                                                    c_p, c_p, c_p, c_size, c_p, c_p, c_p]
        lib.tf_topk_head_loss_grad_bf16_workspace.restype = c_size
        lib.tf_topk_head_loss_grad_bf16_workspace.argtypes = [c_i64, c_i32, c_i64, c_i32]
        lib.tf_topk_route.restype = ctypes.c_int
        lib.tf_topk_route.argtypes = [c_p, c_i32, c_i64, c_i32, c_i64, c_i32, c_p, c_i32, c_i32, c_i32, c_i32, c_i32,
                                      ctypes.c_float, c_p, c_p, c_p, c_p]
        lib.tf_topk_route_grad.restype = ctypes.c_int
        lib.tf_topk_route_grad.argtypes = [c_p, c_i32, c_i64, c_i32, c_i64, c_i32, c_p, c_p, c_i32, c_i32,
                                           ctypes.c_float, c_p, c_p]
        lib.tf_topk_sort_experts.restype = ctypes.c_int
        lib.tf_topk_sort_experts.argtypes = [c_p, c_i64, c_i32, c_i32, c_p, c_size, c_p, c_p, c_p, c_p]
        lib.tf_topk_sort_experts_workspace.restype = c_size
        lib.tf_topk_sort_experts_workspace.argtypes = [c_i64, c_i32, c_i32]
        lib.tf_topk_gather_tokens.restype = ctypes.c_int
        lib.tf_topk_gather_tokens.argtypes = [c_p, c_i32, c_i64, c_i32, c_i64, c_i32, c_p, c_p, c_p, c_p]
        lib.tf_topk_quantize_tokens.restype = ctypes.c_int
        lib.tf_topk_quantize_tokens.argtypes = [c_p, c_i32, c_i64, c_i32, c_i64, c_i32, c_p, c_p, c_p, c_p, c_p]
        lib.tf_topk_combine_tokens.restype = ctypes.c_int
        lib.tf_topk_combine_tokens.argtypes = [c_p, c_i32, c_i64, c_i32, c_i64, c_i32, c_p, c_p, c_p, c_p]
        lib.tf_topk_combine_tokens_grad.restype = ctypes.c_int
        lib.tf_topk_combine_tokens_grad.argtypes = [c_p, c_i32, c_i64, c_i32, c_i64, c_p, c_i64, c_i32, c_p, c_p, c_p,
                                                    c_p, c_p, c_p]
        lib.tf_topk_product_fp8.restype = ctypes.c_int
        lib.tf_topk_product_fp8.argtypes = [c_p, c_p, c_i64, c_i32, c_p, c_p, c_i64, c_i32, c_p, c_i32, c_p, c_p]
        lib.tf_topk_penalize.restype = ctypes.c_int
        lib.tf_topk_penalize.argtypes = [c_p, c_i32, c_i64, c_i64, c_i64, c_p, c_i64, c_i32, c_p, c_p, c_p, c_p, c_p,
                                         c_p, c_p, c_i64, c_i32, c_p, c_i64, c_p, c_i64, c_p]
        lib.tf_topk_strerror.restype = ctypes.c_char_p
        lib.tf_topk_strerror.argtypes = [ctypes.c_int]
        lib.tf_topk_last_cuda_error.restype = ctypes.c_int
        lib.tf_topk_last_cuda_error.argtypes = []
        _lib = lib
    return _lib


def strerror(status: int) -> str:
    return library().tf_topk_strerror(status).decode()


def constants() -> dict:
    lib = library()
    return {
        "max_k": lib.tf_topk_bf16_max_k(),
        "max_spans": lib.tf_topk_bf16_max_spans(),
        "cta_threads": lib.tf_topk_bf16_cta_threads(),
        "chunk_columns": lib.tf_topk_bf16_chunk_columns(),
    }


MAX_K = 64


_raw_stream = None


def _stream_handle(stream, dev) -> int:
    """The cudaStream_t of ``stream``, or of the current stream of ``dev``
    (read through torch's raw-stream query where it has one: a plain
    ``torch.cuda.current_stream`` costs microseconds a call)."""
    global _raw_stream
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        import torch
        f = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _raw_stream = f if f is not None else (lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _raw_stream(dev.index)


def _on_device(dev, fn, *args):
    """fn(*args) with ``dev`` the current CUDA device (the library launches on
    the current device); the device is switched only when it is not already."""
    import torch
    if torch.cuda.current_device() == dev.index:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _check(status: int) -> None:
    if status != OK:
        msg = strerror(status)
        if status == ERR_CUDA:
            msg += f" (cudaError {library().tf_topk_last_cuda_error()})"
        raise TopkError(status, msg)


def tf_topk_bf16(logits: int, rows: int, cols: int, row_stride: int, k: int, out_idx: int,
                 out_val: int, out_count: int, out_nonfinite_mask: int, stream: int | None) -> int:
    """The C entry point with raw pointers (ints); returns the status code."""
    return library().tf_topk_bf16(logits, rows, cols, row_stride, k, out_idx, out_val, out_count,
                                  out_nonfinite_mask, stream)


def tf_topk_bf16_with_plan(logits: int, rows: int, cols: int, row_stride: int, k: int,
                           out_idx: int, out_val: int, out_count: int, out_nonfinite_mask: int,
                           plan: int, stream: int | None) -> int:
    """The C entry point with an explicit launch plan; returns the status code."""
    return library().tf_topk_bf16_with_plan(logits, rows, cols, row_stride, k, out_idx, out_val,
                                            out_count, out_nonfinite_mask, plan, stream)


def tf_topk_bf16_noalloc(logits: int, rows: int, cols: int, row_stride: int, k: int,
                         out_idx: int, out_val: int, out_count: int, out_nonfinite_mask: int,
                         stream: int | None) -> int:
    """The allocation-free C entry point (static scratch shared by every call;
    calls that overlap on the GPU race); returns the status code."""
    return library().tf_topk_bf16_noalloc(logits, rows, cols, row_stride, k, out_idx, out_val,
                                          out_count, out_nonfinite_mask, stream)


def tf_topk_merge_bf16(in_idx: int, in_val: int, in_count: int, in_mask: int, rows: int, shards: int,
                       k_in: int, shard_offset, k: int, out_idx: int, out_val: int, out_count: int,
                       out_mask: int, stream: int | None) -> int:
    """The C merge entry point; `shard_offset` is a host sequence of ints (or
    None to pass NULL).  Returns the status code."""
    off = None
    if shard_offset is not None:
        off = (ctypes.c_int64 * max(1, len(shard_offset)))(*[int(v) for v in shard_offset])
    return library().tf_topk_merge_bf16(in_idx, in_val, in_count, in_mask, rows, shards, k_in, off, k,
                                        out_idx, out_val, out_count, out_mask, stream)


def merge_bf16(idx, val, count, mask, offsets, k: int, *, out=None, stream=None):
    """Merge per-shard top lists into each row's top k.

    idx int32 [shards, rows, k_in], val bf16/int16/uint16 [shards, rows, k_in],
    count int32 [shards, rows], mask int32/uint32 [shards, rows] (all CUDA,
    contiguous), offsets: the column offset of each shard (host ints).
    Returns (idx int32 [rows, k], val [rows, k], count int32 [rows], mask int32 [rows]).
    """
    import torch

    shards, rows, k_in = idx.shape
    for t in (idx, val, count, mask):
        if not t.is_cuda or not t.is_contiguous():
            raise TopkError(ERR_SHAPE, "merge inputs must be contiguous CUDA tensors")
    if out is None:
        dev = idx.device
        out = (torch.empty((rows, k), dtype=torch.int32, device=dev),
               torch.empty((rows, k), dtype=val.dtype, device=dev),
               torch.empty((rows,), dtype=torch.int32, device=dev),
               torch.empty((rows,), dtype=torch.int32, device=dev))
    _check(_on_device(idx.device, tf_topk_merge_bf16, idx.data_ptr(), val.data_ptr(), count.data_ptr(),
                      mask.data_ptr(), rows, shards, k_in, list(offsets), k, out[0].data_ptr(), out[1].data_ptr(),
                      out[2].data_ptr(), out[3].data_ptr(), _stream_handle(stream, idx.device)))
    return out


def tf_topk_nucleus_bf16(val: int, count: int, rows: int, k: int, temperature: float, top_p: float,
                         out_prob: int, out_keep: int, stream: int | None) -> int:
    """The C nucleus (top-p) entry point with raw pointers; returns the status code."""
    return library().tf_topk_nucleus_bf16(val, count, rows, k, temperature, top_p, out_prob, out_keep, stream)


def tf_topk_nucleus(val: int, dtype: int, count: int, rows: int, k: int, temperature: float, top_p: float,
                    out_prob: int, out_keep: int, stream: int | None) -> int:
    """The C nucleus (top-p) entry point for lists of any format; returns the status code."""
    return library().tf_topk_nucleus(val, dtype, count, rows, k, temperature, top_p, out_prob, out_keep, stream)


def nucleus_bf16(val, count, temperature: float, top_p: float, *, out=None, stream=None):
    """Sampling probabilities over top-k lists (softmax of value / T, then the
    shortest best-first prefix with mass >= top_p, renormalised).

    val bf16/int16/uint16 [rows, k] and count int32 [rows] as ``topk_bf16``
    returns them (contiguous CUDA tensors).  Returns (prob float32 [rows, k],
    keep int32 [rows]).
    """
    return nucleus(val, count, temperature, top_p, dtype=DTYPE_BF16, out=out, stream=stream)


def nucleus(val, count, temperature: float, top_p: float, *, dtype: int | None = None, out=None, stream=None):
    """``nucleus_bf16`` for lists of any format ``select_topk`` returns:
    val bfloat16 / float16 / float32 [rows, k] (or int16 / int32 bits with
    ``dtype``), count int32 [rows]."""
    import torch

    codes = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16, torch.float32: DTYPE_F32,
             torch.int16: DTYPE_BF16, torch.uint16: DTYPE_BF16, torch.int32: DTYPE_F32}
    if dtype is None:
        if val.dtype not in codes:
            raise TypeError(f"unsupported list dtype {val.dtype}")
        dtype = codes[val.dtype]
    if val.element_size() != (4 if dtype == DTYPE_F32 else 2):
        raise TypeError("element size does not match dtype")
    if val.dim() != 2 or count.dim() != 1 or count.shape[0] != val.shape[0]:
        raise ValueError("val must be [rows, k] and count [rows]")
    for t in (val, count):
        if not t.is_cuda or not t.is_contiguous():
            raise TopkError(ERR_SHAPE, "nucleus inputs must be contiguous CUDA tensors")
    rows, k = val.shape
    if out is None:
        out = (torch.empty((rows, k), dtype=torch.float32, device=val.device),
               torch.empty((rows,), dtype=torch.int32, device=val.device))
    _check(_on_device(val.device, tf_topk_nucleus, val.data_ptr(), dtype, count.data_ptr(), rows, k,
                      float(temperature), float(top_p), out[0].data_ptr(), out[1].data_ptr(),
                      _stream_handle(stream, val.device)))
    return out


def tf_topk_select(logits: int, dtype: int, rows: int, cols: int, row_stride: int, k: int, out_idx: int,
                   out_val: int, out_count: int, out_nonfinite_mask: int, stream: int | None) -> int:
    """The C entry point for bf16 / fp16 / fp32 rows and k up to 1024; returns the status code."""
    return library().tf_topk_select(logits, dtype, rows, cols, row_stride, k, out_idx, out_val, out_count,
                                    out_nonfinite_mask, stream)


def tf_topk_select_with_plan(logits: int, dtype: int, rows: int, cols: int, row_stride: int, k: int,
                             out_idx: int, out_val: int, out_count: int, out_nonfinite_mask: int, plan: int,
                             stream: int | None) -> int:
    """tf_topk_select with a plan (0 AUTO, PLAN_WIDE, or a bf16 plan for k <= 64)."""
    return library().tf_topk_select_with_plan(logits, dtype, rows, cols, row_stride, k, out_idx, out_val,
                                              out_count, out_nonfinite_mask, plan, stream)


def select_topk(x, k: int, *, dtype: int | None = None, plan: int = 0, out=None, stream=None):
    """Exact top-k of every row of a CUDA bf16 / fp16 / fp32 matrix, k up to 1024.

    ``x``: bfloat16, float16 or float32 (or int16 / int32 holding the bits,
    with ``dtype`` one of DTYPE_*), 1-D or 2-D with unit column stride.
    Returns ``(idx int32[rows,k], val[rows,k] (x's dtype), count int32[rows],
    mask int32[rows])``.
    """
    import torch

    codes = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16, torch.float32: DTYPE_F32}
    if not x.is_cuda:
        raise ValueError("select_topk needs a CUDA tensor (no CPU path exists)")
    if dtype is None:
        if x.dtype not in codes:
            raise TypeError(f"pass dtype= for a {x.dtype} tensor of bits")
        dtype = codes[x.dtype]
    if x.element_size() != (4 if dtype == DTYPE_F32 else 2):
        raise TypeError("element size does not match dtype")
    if x.dim() == 1:
        x = x.unsqueeze(0)
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be 1-D or 2-D with contiguous columns")
    rows, cols = x.shape
    row_stride = x.stride(0) if rows > 1 else max(cols, x.stride(0))
    dev = x.device
    if out is None:
        out = (torch.empty((rows, k), dtype=torch.int32, device=dev),
               torch.empty((rows, k), dtype=x.dtype, device=dev),
               torch.empty((rows,), dtype=torch.int32, device=dev),
               torch.empty((rows,), dtype=torch.int32, device=dev))
    _check(_on_device(dev, tf_topk_select_with_plan, x.data_ptr(), dtype, rows, cols, row_stride, k,
                      out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(), plan,
                      _stream_handle(stream, dev)))
    return out


HEAD_MAX_ROWS = 16


def tf_topk_head_bf16(hidden: int, weight: int, rows: int, dim: int, vocab: int, k: int, workspace: int,
                      workspace_bytes: int, out_idx: int, out_val: int, out_count: int, out_mask: int,
                      stream: int | None) -> int:
    """The fused draft-head entry point with raw pointers; returns the status code."""
    return library().tf_topk_head_bf16(hidden, weight, rows, dim, vocab, k, workspace, workspace_bytes, out_idx,
                                       out_val, out_count, out_mask, stream)


def tf_topk_head_bf16_workspace(rows: int, k: int) -> int:
    """Workspace bytes tf_topk_head_bf16 needs on the current device (0 for bad arguments)."""
    return library().tf_topk_head_bf16_workspace(rows, k)


def head_topk_bf16(hidden, weight, k: int, *, out=None, workspace=None, stream=None):
    """Top-k of every row of the draft head's logits, bf16(hidden @ weight.T),
    computed and selected in one kernel (the logits are never stored).

    ``hidden``: CUDA bf16 (or int16 bits) [rows, dim], rows <= 16;
    ``weight``: CUDA bf16 (or int16 bits) [vocab, dim]; both contiguous.
    Returns ``(idx int32[rows,k], val bfloat16[rows,k], count int32[rows],
    mask int32[rows])`` as ``topk_bf16`` gives them for the logit matrix.
    ``workspace``: a CUDA uint8 tensor of at least
    ``tf_topk_head_bf16_workspace(rows, k)`` bytes (allocated here if None).
    """
    import torch

    for t in (hidden, weight):
        if not t.is_cuda or not t.is_contiguous() or t.dim() != 2:
            raise ValueError("hidden and weight must be contiguous 2-D CUDA tensors")
        if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
            raise TypeError(f"expected bf16 bits, got {t.dtype}")
    rows, dim = hidden.shape
    vocab = weight.shape[0]
    if weight.shape[1] != dim:
        raise ValueError("hidden and weight disagree on dim")
    dev = hidden.device
    if out is None:
        out = (torch.empty((rows, k), dtype=torch.int32, device=dev),
               torch.empty((rows, k), dtype=torch.bfloat16, device=dev),
               torch.empty((rows,), dtype=torch.int32, device=dev),
               torch.empty((rows,), dtype=torch.int32, device=dev))
    if workspace is None:
        need = _on_device(dev, tf_topk_head_bf16_workspace, rows, k) if 1 <= rows <= HEAD_MAX_ROWS else 0
        workspace = torch.empty((max(need, 8),), dtype=torch.uint8, device=dev)
    _check(_on_device(dev, tf_topk_head_bf16, hidden.data_ptr(), weight.data_ptr(), rows, dim, vocab, k,
                      workspace.data_ptr(), workspace.numel(), out[0].data_ptr(), out[1].data_ptr(),
                      out[2].data_ptr(), out[3].data_ptr(), _stream_handle(stream, dev)))
    return out


def tf_topk_head_loss_bf16(hidden: int, hidden_stride: int, weight: int, weight_stride: int, rows: int, dim: int,
                           vocab: int, target: int, target_bytes: int, ignore_index: int, workspace: int,
                           workspace_bytes: int, out_loss: int, out_lse: int, stream: int | None) -> int:
    """The C entry point of the head's loss with raw pointers; returns the status code."""
    return library().tf_topk_head_loss_bf16(hidden, hidden_stride, weight, weight_stride, rows, dim, vocab, target,
                                            target_bytes, ignore_index, workspace, workspace_bytes, out_loss, out_lse,
                                            stream)


def tf_topk_head_loss_bf16_workspace(rows: int, dim: int, vocab: int) -> int:
    """Workspace bytes tf_topk_head_loss_bf16 needs on the current device (0 for bad arguments)."""
    return library().tf_topk_head_loss_bf16_workspace(rows, dim, vocab)


def tf_topk_head_loss_grad_bf16(hidden: int, hidden_stride: int, weight: int, weight_stride: int, rows: int, dim: int,
                                vocab: int, target: int, target_bytes: int, ignore_index: int, lse: int,
                                grad_loss: int, workspace: int, workspace_bytes: int, out_grad_hidden: int | None,
                                out_grad_weight: int | None, stream: int | None) -> int:
    """The C entry point of the head loss's gradient with raw pointers; returns the status code."""
    return library().tf_topk_head_loss_grad_bf16(hidden, hidden_stride, weight, weight_stride, rows, dim, vocab,
                                                 target, target_bytes, ignore_index, lse, grad_loss, workspace,
                                                 workspace_bytes, out_grad_hidden, out_grad_weight, stream)


def tf_topk_head_loss_grad_bf16_workspace(rows: int, dim: int, vocab: int, least: bool = False) -> int:
    """Workspace bytes tf_topk_head_loss_grad_bf16 makes good use of on the
    current device, or the least it accepts (0 for bad arguments)."""
    return library().tf_topk_head_loss_grad_bf16_workspace(rows, dim, vocab, int(least))


_torch = None


def _need_torch():
    """The torch module (imported on the first tensor-level call)."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _head_inputs(hidden, weight, target):
    """(rows, dim, vocab, hidden row stride, weight row stride) of a head's loss, checked."""
    torch = _torch or _need_torch()
    for name, t in (("hidden", hidden), ("weight", weight)):
        if t.dtype is not torch.bfloat16 and t.dtype not in (torch.int16, torch.uint16):
            raise TypeError(f"expected bf16 bits, got {t.dtype}")
        if not t.is_cuda or t.dim() != 2:
            raise ValueError(f"{name} must be a 2-D CUDA tensor")
    rows, dim = hidden.shape
    vocab, width = weight.shape
    hs, ws = hidden.stride(), weight.stride()
    if width != dim:
        raise ValueError("hidden and weight disagree on dim")
    if dim > 1 and (hs[1] != 1 or ws[1] != 1):
        raise ValueError("hidden and weight must have contiguous columns")
    if target.dtype is not torch.int64 and target.dtype is not torch.int32:
        raise TypeError(f"target must be int64 or int32, got {target.dtype}")
    if target.shape != (rows,) or not target.is_contiguous():
        raise ValueError("target must be a contiguous [rows] tensor")
    dev = hidden.device
    if weight.device != dev or target.device != dev:
        raise ValueError("hidden, weight and target must be on one device")
    round_up = -(-dim // 8) * 8  # the stride of a single row is free
    return rows, dim, vocab, hs[0] if rows > 1 else round_up, ws[0] if vocab > 1 else round_up


def _check_out(t, shape, dtype, dev, name):
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on the inputs' device")


def _empty(shape, dtype, dev, stream):
    """A fresh tensor whose memory belongs to the stream the call runs on: what
    is freed there may still be in use by the work queued before it, and what a
    call frees at its end (a workspace) is reused by the work after it."""
    torch = _torch or _need_torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _workspace(workspace, need, args, dev, stream):
    """A caller's workspace, checked, or a fresh one of need(*args) bytes."""
    if workspace is None:
        return _empty((need(*args) or 8,), _torch.uint8, dev, stream)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return workspace


def head_loss_bf16(hidden, weight, target, *, ignore_index: int = -100, out=None, workspace=None, stream=None):
    """Softmax cross entropy of the head's logits ``hidden @ weight.T`` (bf16
    in, fp32 sums, not rounded) against one target column per row, without
    storing the logits.

    ``hidden``: CUDA bf16 (or int16 bits) [rows, dim], ``weight`` [vocab, dim],
    both with contiguous columns, dim and row strides multiples of 8;
    ``target``: int64 or int32 [rows].
    Returns ``(loss float32[rows], lse float32[rows])``: per row, 0 and 0 where
    the target is ``ignore_index``, NaN where it is any other value outside the
    vocabulary.  ``loss`` is not reduced; ``lse`` is what
    ``head_loss_grad_bf16`` takes.  ``out`` may supply those two tensors and
    ``workspace`` a CUDA tensor of at least
    ``tf_topk_head_loss_bf16_workspace(rows, dim, vocab)`` bytes.
    """
    rows, dim, vocab, hs, ws = _head_inputs(hidden, weight, target)
    torch, dev = _torch, hidden.device
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return head_loss_bf16(hidden, weight, target, ignore_index=ignore_index, out=out, workspace=workspace,
                                  stream=stream)
    if out is None:
        loss, lse = _empty((rows,), torch.float32, dev, stream), _empty((rows,), torch.float32, dev, stream)
    else:
        loss, lse = out
        _check_out(loss, (rows,), torch.float32, dev, "loss")
        _check_out(lse, (rows,), torch.float32, dev, "lse")
    lib = _lib or library()
    space = _workspace(workspace, lib.tf_topk_head_loss_bf16_workspace, (rows, dim, vocab), dev, stream)
    _check(lib.tf_topk_head_loss_bf16(hidden.data_ptr(), hs, weight.data_ptr(), ws, rows, dim, vocab,
                                      target.data_ptr(), target.element_size(), ignore_index, space.data_ptr(),
                                      space.nbytes, loss.data_ptr(), lse.data_ptr(), _stream_handle(stream, dev)))
    return loss, lse


def head_loss_grad_bf16(hidden, weight, target, lse, grad_loss, *, ignore_index: int = -100, hidden_grad: bool = True,
                        weight_grad: bool = True, out=None, workspace=None, stream=None):
    """Gradient of ``head_loss_bf16``: with ``grad_loss`` float32 [rows] the
    gradient of its losses and ``lse`` as it returned it, gives
    ``(grad_hidden bf16[rows, dim], grad_weight bf16[vocab, dim])``.

    The logits are computed again, in pieces of the vocabulary.  A gradient
    that is not wanted (``hidden_grad`` / ``weight_grad`` False) is not
    computed and None in its place.  Rows that do not count get zeros and
    reach nothing, whatever they hold.  ``out`` may supply the two tensors
    (None for one not wanted) and ``workspace`` a CUDA tensor of any size from
    ``tf_topk_head_loss_grad_bf16_workspace(rows, dim, vocab, True)`` bytes on.
    """
    rows, dim, vocab, hs, ws = _head_inputs(hidden, weight, target)
    torch, dev = _torch, hidden.device
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return head_loss_grad_bf16(hidden, weight, target, lse, grad_loss, ignore_index=ignore_index,
                                       hidden_grad=hidden_grad, weight_grad=weight_grad, out=out, workspace=workspace,
                                       stream=stream)
    _check_out(lse, (rows,), torch.float32, dev, "lse")
    _check_out(grad_loss, (rows,), torch.float32, dev, "grad_loss")
    if not hidden_grad and not weight_grad:
        return None, None
    if out is None:
        dh = _empty((rows, dim), torch.bfloat16, dev, stream) if hidden_grad else None
        dw = _empty((vocab, dim), torch.bfloat16, dev, stream) if weight_grad else None
    else:
        dh, dw = out[0] if hidden_grad else None, out[1] if weight_grad else None
        if hidden_grad:
            _check_out(dh, (rows, dim), torch.bfloat16, dev, "grad_hidden")
        if weight_grad:
            _check_out(dw, (vocab, dim), torch.bfloat16, dev, "grad_weight")
    lib = _lib or library()
    space = _workspace(workspace, lib.tf_topk_head_loss_grad_bf16_workspace, (rows, dim, vocab, 0), dev, stream)
    _check(lib.tf_topk_head_loss_grad_bf16(hidden.data_ptr(), hs, weight.data_ptr(), ws, rows, dim, vocab,
                                           target.data_ptr(), target.element_size(), ignore_index, lse.data_ptr(),
                                           grad_loss.data_ptr(), space.data_ptr(), space.nbytes,
                                           dh.data_ptr() if hidden_grad else None,
                                           dw.data_ptr() if weight_grad else None, _stream_handle(stream, dev)))
    return dh, dw


ROUTE_SCORES = {"softmax": 0, "sigmoid": 1}
ROUTE_MAX_EXPERTS, ROUTE_MAX_K, ROUTE_MAX_GROUPS = 1024, 32, 32


def tf_topk_route(logits: int, dtype: int, tokens: int, experts: int, row_stride: int, k: int, bias: int | None,
                  score: int, groups: int, groups_kept: int, group_best: int, renormalize: int, scale: float,
                  out_idx: int, out_weight: int, load: int | None, stream: int | None) -> int:
    """The C entry point of expert routing with raw pointers; returns the status code."""
    return library().tf_topk_route(logits, dtype, tokens, experts, row_stride, k, bias, score, groups, groups_kept,
                                   group_best, renormalize, scale, out_idx, out_weight, load, stream)


def tf_topk_route_grad(logits: int, dtype: int, tokens: int, experts: int, row_stride: int, k: int, idx: int,
                       grad_weight: int, score: int, renormalize: int, scale: float, out_grad_logits: int,
                       stream: int | None) -> int:
    """The C entry point of the routing gradient with raw pointers; returns the status code."""
    return library().tf_topk_route_grad(logits, dtype, tokens, experts, row_stride, k, idx, grad_weight, score,
                                        renormalize, scale, out_grad_logits, stream)


_logit_codes = None


def _router_logits(logits, score: str):
    """(dtype code, tokens, experts, row stride, score code) of a router's logits, checked."""
    global _logit_codes
    if _logit_codes is None:
        torch = _need_torch()
        _logit_codes = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16, torch.float32: DTYPE_F32}
    code, how = _logit_codes.get(logits.dtype), ROUTE_SCORES.get(score)
    if code is None:
        raise TypeError(f"logits must be bfloat16, float16 or float32, got {logits.dtype}")
    if how is None:
        raise ValueError(f"score must be one of {tuple(ROUTE_SCORES)}, got {score!r}")
    if not logits.is_cuda or logits.dim() != 2:
        raise ValueError("logits must be a 2-D CUDA tensor")
    tokens, experts = logits.shape
    stride = logits.stride()
    if experts > 1 and stride[1] != 1:
        raise ValueError("logits must have contiguous columns")
    return code, tokens, experts, stride[0] if tokens > 1 else experts, how


def route_experts(logits, k: int, *, bias=None, score: str = "softmax", groups: int = 1, groups_kept: int | None = None,
                  group_best: int = 2, renormalize: bool = True, scale: float = 1.0, load=None, out=None, stream=None):
    """Each token's best ``k`` experts, best first (ties to the lower expert),
    with their weights.

    ``logits``: CUDA bf16 / fp16 / fp32 [tokens, experts], contiguous columns.
    Scores are the sigmoid or the softmax of the logits; an expert whose logit
    is NaN or -inf is out of reach.  ``bias`` (float32 [experts]) moves the
    choice only.  With ``groups`` > 1 only the experts of the ``groups_kept``
    best groups remain, a group's value being the sum of its best
    ``group_best`` (1 or 2) choices.  Weights are the chosen scores, with
    ``renormalize`` over their sum, times ``scale``.
    Returns ``(idx int32[tokens, k], weight float32[tokens, k])``; places that
    no expert is left for hold -1 and 0.  ``load`` (int32 [experts]), if given,
    grows by the tokens each expert was chosen for.  ``out`` may supply idx and
    weight.
    """
    code, tokens, experts, stride, how = _router_logits(logits, score)
    torch, dev = _torch, logits.device
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return route_experts(logits, k, bias=bias, score=score, groups=groups, groups_kept=groups_kept,
                                 group_best=group_best, renormalize=renormalize, scale=scale, load=load, out=out,
                                 stream=stream)
    if bias is not None:
        _check_out(bias, (experts,), torch.float32, dev, "bias")
    if load is not None:
        _check_out(load, (experts,), torch.int32, dev, "load")
    if out is None:
        # a bad k is the library's to refuse
        shape = (tokens, k if k > 0 else 0)
        idx, weight = _empty(shape, torch.int32, dev, stream), _empty(shape, torch.float32, dev, stream)
    else:
        idx, weight = out
        _check_out(idx, (tokens, k), torch.int32, dev, "idx")
        _check_out(weight, (tokens, k), torch.float32, dev, "weight")
    _check((_lib or library()).tf_topk_route(
        logits.data_ptr(), code, tokens, experts, stride, k, None if bias is None else bias.data_ptr(), how, groups,
        groups if groups_kept is None else groups_kept, group_best, bool(renormalize), scale, idx.data_ptr(),
        weight.data_ptr(), None if load is None else load.data_ptr(), _stream_handle(stream, dev)))
    return idx, weight


def route_experts_grad(logits, idx, grad_weight, *, score: str = "softmax", renormalize: bool = True,
                       scale: float = 1.0, out=None, stream=None):
    """Gradient of ``route_experts``'s weights for the logits, the choice held
    fixed: ``idx`` int32 [tokens, k] as it returned it, ``grad_weight`` float32
    [tokens, k], the other arguments as in its call.  Returns the gradient
    [tokens, experts] in the logits' dtype (zero where nothing flows)."""
    code, tokens, experts, stride, how = _router_logits(logits, score)
    torch, dev = _torch, logits.device
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return route_experts_grad(logits, idx, grad_weight, score=score, renormalize=renormalize, scale=scale,
                                      out=out, stream=stream)
    if idx.dim() != 2 or idx.shape[0] != tokens:
        raise ValueError("idx must be [tokens, k]")
    k = idx.shape[1]
    _check_out(idx, (tokens, k), torch.int32, dev, "idx")
    _check_out(grad_weight, (tokens, k), torch.float32, dev, "grad_weight")
    if out is None:
        out = _empty((tokens, experts), logits.dtype, dev, stream)
    else:
        _check_out(out, (tokens, experts), logits.dtype, dev, "out")
    _check((_lib or library()).tf_topk_route_grad(
        logits.data_ptr(), code, tokens, experts, stride, k, idx.data_ptr(), grad_weight.data_ptr(), how,
        bool(renormalize), scale, out.data_ptr(), _stream_handle(stream, dev)))
    return out


# Sizes that the C calls take as int32 are held against it here: ctypes would hand
# over the low bits of a larger one, which may be a size that runs.
_INT32_MAX = 2**31 - 1


class ExpertOrder(NamedTuple):
    """The order of routing's choices by expert, as ``sort_by_expert`` gives it."""

    slot: Any  # int32 [tokens, k]: the place of each choice, -1 for one that takes no part
    source: Any  # int32 [tokens * k]: the choice (t * k + j) at each place, -1 behind the last
    offsets: Any  # int32 [experts + 1]: the first place of each expert, and the end of the last


def tf_topk_sort_experts(idx: int, tokens: int, k: int, experts: int, workspace: int | None, workspace_bytes: int,
                         out_slot: int, out_source: int, out_offsets: int, stream: int | None) -> int:
    """The C entry point of the sort by expert with raw pointers; returns the status code."""
    return library().tf_topk_sort_experts(idx, tokens, k, experts, workspace, workspace_bytes, out_slot, out_source,
                                          out_offsets, stream)


def tf_topk_sort_experts_workspace(tokens: int, k: int, experts: int) -> int:
    """Workspace bytes tf_topk_sort_experts needs on the current device (0 where it needs none)."""
    return library().tf_topk_sort_experts_workspace(tokens, k, experts)


def sort_by_expert(idx, experts: int, *, out=None, workspace=None, stream=None) -> ExpertOrder:
    """Order of ``route_experts``'s choices by expert, and by token and place
    within an expert (a stable sort).

    ``idx``: CUDA int32 [tokens, k], contiguous; choices outside
    [0, ``experts``) take no part.  Returns an ``ExpertOrder``.  ``out`` may
    supply its three tensors, ``workspace`` a CUDA tensor of at least
    ``tf_topk_sort_experts_workspace(tokens, k, experts)`` bytes.
    """
    torch = _torch or _need_torch()
    if idx.dtype is not torch.int32:
        raise TypeError(f"idx must be int32, got {idx.dtype}")
    if not idx.is_cuda or idx.dim() != 2 or not idx.is_contiguous():
        raise ValueError("idx must be a contiguous 2-D CUDA tensor")
    dev = idx.device
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return sort_by_expert(idx, experts, out=out, workspace=workspace, stream=stream)
    tokens, k = idx.shape
    if k > _INT32_MAX:
        _check(ERR_K)
    if not -_INT32_MAX <= experts <= _INT32_MAX:
        _check(ERR_SHAPE)
    n = tokens * k
    if out is None:
        # a bad count of experts is the library's to refuse
        order = ExpertOrder(_empty((tokens, k), torch.int32, dev, stream), _empty((n,), torch.int32, dev, stream),
                            _empty((max(experts, 0) + 1,), torch.int32, dev, stream))
    else:
        order = ExpertOrder(*out)
        _check_out(order.slot, (tokens, k), torch.int32, dev, "slot")
        _check_out(order.source, (n,), torch.int32, dev, "source")
        _check_out(order.offsets, (experts + 1,), torch.int32, dev, "offsets")
    lib = _lib or library()
    space, room = None, 0
    if workspace is not None:
        space = _workspace(workspace, None, (), dev, stream)
    elif lib.tf_topk_sort_experts_workspace(tokens, k, experts):
        space = _workspace(None, lib.tf_topk_sort_experts_workspace, (tokens, k, experts), dev, stream)
    if space is not None:
        room, space_ptr = space.nbytes, space.data_ptr()
    else:
        space_ptr = None
    _check(lib.tf_topk_sort_experts(idx.data_ptr(), tokens, k, experts, space_ptr, room, order.slot.data_ptr(),
                                    order.source.data_ptr(), order.offsets.data_ptr(), _stream_handle(stream, dev)))
    return order


def _rows_code(x, name):
    """(dtype code, rows, dim, row stride) of a matrix of rows, checked."""
    global _logit_codes
    if _logit_codes is None:
        torch = _need_torch()
        _logit_codes = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16, torch.float32: DTYPE_F32}
    code = _logit_codes.get(x.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {x.dtype}")
    if not x.is_cuda or x.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    rows, dim = x.shape
    stride = x.stride()
    if dim > 1 and stride[1] != 1:
        raise ValueError(f"{name} must have contiguous columns")
    if dim > _INT32_MAX:
        _check(ERR_SHAPE)
    return code, rows, dim, stride[0] if rows > 1 else dim


def _order_of(order, tokens, dev):
    """(slot, source, k) of an order for so many tokens, checked."""
    slot, source = order[0], order[1]
    if slot.dim() != 2 or slot.shape[0] != tokens:
        raise ValueError("the order is not of this many tokens")
    k = slot.shape[1]
    if k > _INT32_MAX:
        _check(ERR_K)
    _check_out(slot, (tokens, k), _torch.int32, dev, "slot")
    _check_out(source, (tokens * k,), _torch.int32, dev, "source")
    return slot, source, k


def tf_topk_gather_tokens(x: int, dtype: int, tokens: int, dim: int, row_stride: int, k: int, slot: int, source: int,
                          out_rows: int, stream: int | None) -> int:
    """The C entry point of the gather by expert with raw pointers; returns the status code."""
    return library().tf_topk_gather_tokens(x, dtype, tokens, dim, row_stride, k, slot, source, out_rows, stream)


def gather_tokens(x, order: ExpertOrder, *, out=None, stream=None):
    """The tokens' rows in the order of ``sort_by_expert``: a row for each
    choice, zeros behind the last.  ``x``: CUDA bf16 / fp16 / fp32
    [tokens, dim], contiguous columns.  Returns [tokens * k, dim] of its dtype."""
    code, tokens, dim, stride = _rows_code(x, "x")
    torch, dev = _torch, x.device
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return gather_tokens(x, order, out=out, stream=stream)
    slot, source, k = _order_of(order, tokens, dev)
    if out is None:
        out = _empty((tokens * k, dim), x.dtype, dev, stream)
    else:
        _check_out(out, (tokens * k, dim), x.dtype, dev, "out")
    _check((_lib or library()).tf_topk_gather_tokens(x.data_ptr(), code, tokens, dim, stride, k, slot.data_ptr(),
                                                     source.data_ptr(), out.data_ptr(), _stream_handle(stream, dev)))
    return out


def tf_topk_combine_tokens(rows: int, dtype: int, tokens: int, dim: int, row_stride: int, k: int, slot: int,
                           weight: int | None, out: int, stream: int | None) -> int:
    """The C entry point of the experts' rows combined by token; returns the status code."""
    return library().tf_topk_combine_tokens(rows, dtype, tokens, dim, row_stride, k, slot, weight, out, stream)


def combine_tokens(rows, order: ExpertOrder, weight=None, *, out=None, stream=None):
    """The experts' rows back to their tokens: out[t] = sum over j of
    weight[t, j] * rows[slot[t, j]], in 32 bits, rounded once.

    ``rows``: CUDA bf16 / fp16 / fp32 [tokens * k, dim], contiguous columns;
    ``weight``: float32 [tokens, k] as ``route_experts`` returns it, or None
    for plain sums.  Choices without a place are left out, whatever their
    weight.  Returns [tokens, dim] of the rows' dtype.
    """
    code, n, dim, stride = _rows_code(rows, "rows")
    torch, dev = _torch, rows.device
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return combine_tokens(rows, order, weight, out=out, stream=stream)
    tokens = order[0].shape[0]
    slot, _, k = _order_of(order, tokens, dev)
    if n != tokens * k:
        raise ValueError("rows must have one row for each choice")
    if weight is not None:
        _check_out(weight, (tokens, k), torch.float32, dev, "weight")
    if out is None:
        out = _empty((tokens, dim), rows.dtype, dev, stream)
    else:
        _check_out(out, (tokens, dim), rows.dtype, dev, "out")
    _check((_lib or library()).tf_topk_combine_tokens(
        rows.data_ptr(), code, tokens, dim, stride, k, slot.data_ptr(), None if weight is None else weight.data_ptr(),
        out.data_ptr(), _stream_handle(stream, dev)))
    return out


def gather_tokens_grad(grad_rows, order: ExpertOrder, *, out=None, stream=None):
    """Gradient of ``gather_tokens`` for x: each token's sum over its rows of
    ``grad_rows`` [tokens * k, dim], in 32 bits, rounded once."""
    return combine_tokens(grad_rows, order, None, out=out, stream=stream)


def tf_topk_combine_tokens_grad(grad_out: int, dtype: int, tokens: int, dim: int, grad_stride: int, rows: int,
                                row_stride: int, k: int, slot: int, source: int, weight: int, out_grad_rows: int,
                                out_grad_weight: int, stream: int | None) -> int:
    """The C entry point of the gradient of tf_topk_combine_tokens; returns the status code."""
    return library().tf_topk_combine_tokens_grad(grad_out, dtype, tokens, dim, grad_stride, rows, row_stride, k, slot,
                                                 source, weight, out_grad_rows, out_grad_weight, stream)


def combine_tokens_grad(grad_out, rows, order: ExpertOrder, weight, *, out=None, stream=None):
    """Gradient of ``combine_tokens``: with ``grad_out`` [tokens, dim] (the
    rows' dtype) gives ``(grad_rows [tokens * k, dim], grad_weight float32
    [tokens, k])``; rows behind the last place and choices without one get 0."""
    code, tokens, dim, grad_stride = _rows_code(grad_out, "grad_out")
    torch, dev = _torch, grad_out.device
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return combine_tokens_grad(grad_out, rows, order, weight, out=out, stream=stream)
    slot, source, k = _order_of(order, tokens, dev)
    _, n, width, row_stride = _rows_code(rows, "rows")
    if n != tokens * k or width != dim or rows.dtype is not grad_out.dtype or rows.device != dev:
        raise ValueError("rows must have one row for each choice, of grad_out's dim, dtype and device")
    _check_out(weight, (tokens, k), torch.float32, dev, "weight")
    if out is None:
        grad_rows = _empty((n, dim), rows.dtype, dev, stream)
        grad_weight = _empty((tokens, k), torch.float32, dev, stream)
    else:
        grad_rows, grad_weight = out
        _check_out(grad_rows, (n, dim), rows.dtype, dev, "grad_rows")
        _check_out(grad_weight, (tokens, k), torch.float32, dev, "grad_weight")
    _check((_lib or library()).tf_topk_combine_tokens_grad(
        grad_out.data_ptr(), code, tokens, dim, grad_stride, rows.data_ptr(), row_stride, k, slot.data_ptr(),
        source.data_ptr(), weight.data_ptr(), grad_rows.data_ptr(), grad_weight.data_ptr(),
        _stream_handle(stream, dev)))
    return grad_rows, grad_weight


FP8_BLOCK = 128


def tf_topk_quantize_tokens(x: int, dtype: int, tokens: int, dim: int, row_stride: int, k: int, slot: int | None,
                            source: int | None, out_q: int, out_scale: int, stream: int | None) -> int:
    """The C entry point of rows in 8 bits with raw pointers; returns the status code."""
    return library().tf_topk_quantize_tokens(x, dtype, tokens, dim, row_stride, k, slot, source, out_q, out_scale,
                                             stream)


def quantize_tokens_fp8(x, order: ExpertOrder | None = None, *, out=None, stream=None):
    """Rows in 8 bits: e4m3 values with a scale for each 128 of a row, the
    scale being the largest magnitude (2^-100 at least) times 1/448 in 32 bits.

    ``x``: CUDA bf16 / fp16 / fp32 [tokens, dim], contiguous columns, dim a
    multiple of 16.  With ``order`` the rows come in the order of
    ``sort_by_expert`` (zeros behind the last place).  Returns ``(q
    float8_e4m3fn [rows, dim], scale float32 [rows, ceil(dim / 128)])`` for
    ``product_fp8``.
    """
    code, tokens, dim, stride = _rows_code(x, "x")
    torch, dev = _torch, x.device
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return quantize_tokens_fp8(x, order, out=out, stream=stream)
    slot, source, k = (None, None, 1) if order is None else _order_of(order, tokens, dev)
    rows, blocks = tokens * k, -(-dim // FP8_BLOCK)
    if out is None:
        q = _empty((rows, dim), torch.float8_e4m3fn, dev, stream)
        scale = _empty((rows, blocks), torch.float32, dev, stream)
    else:
        q, scale = out
        _check_out(q, (rows, dim), torch.float8_e4m3fn, dev, "q")
        _check_out(scale, (rows, blocks), torch.float32, dev, "scale")
    _check((_lib or library()).tf_topk_quantize_tokens(
        x.data_ptr(), code, tokens, dim, stride, k, None if slot is None else slot.data_ptr(),
        None if source is None else source.data_ptr(), q.data_ptr(), scale.data_ptr(), _stream_handle(stream, dev)))
    return q, scale


def tf_topk_product_fp8(q: int, scale: int, rows: int, dim: int, weight: int, weight_scale: int, cols: int,
                        groups: int, offsets: int | None, dtype: int, out: int, stream: int | None) -> int:
    """The C entry point of the product in 8 bits with raw pointers; returns the status code."""
    return library().tf_topk_product_fp8(q, scale, rows, dim, weight, weight_scale, cols, groups, offsets, dtype, out,
                                         stream)


def product_fp8(q, scale, weight, weight_scale, *, offsets=None, dtype=None, out=None, stream=None):
    """Product of rows in 8 bits with weights in 8 bits, of one matrix or of
    the experts' matrices over their sorted rows; 32-bit sums, each block of
    128 dims scaled as it is added.

    ``q`` float8_e4m3fn [rows, dim] and ``scale`` float32 [rows,
    ceil(dim / 128)] as ``quantize_tokens_fp8`` returns them; ``weight``
    float8_e4m3fn [cols, dim] with ``weight_scale`` float32 [ceil(cols / 128),
    ceil(dim / 128)], or with ``offsets`` (int32 [experts + 1], ascending from
    0, as in an ``ExpertOrder``) [experts, cols, dim] and [experts, ...].  All
    contiguous, dim a multiple of 16.  Returns [rows, cols] of ``dtype``
    (bfloat16, float16 or float32; bfloat16 if None); rows behind the last
    expert's become zeros.
    """
    torch = _torch or _need_torch()
    f8 = torch.float8_e4m3fn
    if q.dtype is not f8 or weight.dtype is not f8:
        raise TypeError(f"q and weight must be float8_e4m3fn, got {q.dtype} and {weight.dtype}")
    if not q.is_cuda or q.dim() != 2 or not q.is_contiguous():
        raise ValueError("q must be a contiguous 2-D CUDA tensor")
    dev = q.device
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return product_fp8(q, scale, weight, weight_scale, offsets=offsets, dtype=dtype, out=out, stream=stream)
    rows, dim = q.shape
    shape = weight.shape
    if offsets is None:
        shape = (1, *shape)
    if len(shape) != 3 or shape[2] != dim:
        raise ValueError("weight must be [cols, dim], or with offsets [experts, cols, dim]")
    groups, cols = shape[0], shape[1]
    if dim > _INT32_MAX or groups > _INT32_MAX:
        _check(ERR_SHAPE)
    blocks, col_blocks = -(-dim // FP8_BLOCK), -(-cols // FP8_BLOCK)
    _check_out(weight, tuple(weight.shape), f8, dev, "weight")
    _check_out(scale, (rows, blocks), torch.float32, dev, "scale")
    _check_out(weight_scale, (col_blocks, blocks) if offsets is None else (groups, col_blocks, blocks), torch.float32,
               dev, "weight_scale")
    if offsets is not None:
        _check_out(offsets, (groups + 1,), torch.int32, dev, "offsets")
    if out is None:
        out = _empty((rows, cols), dtype or torch.bfloat16, dev, stream)
    else:
        _check_out(out, (rows, cols), dtype or out.dtype, dev, "out")
    code = _rows_code(out, "out")[0]
    _check((_lib or library()).tf_topk_product_fp8(
        q.data_ptr(), scale.data_ptr(), rows, dim, weight.data_ptr(), weight_scale.data_ptr(), cols, groups,
        None if offsets is None else offsets.data_ptr(), code, out.data_ptr(), _stream_handle(stream, dev)))
    return out


PENALTY_MAX_BIASES = 65535


def tf_topk_penalize(logits: int, dtype: int, rows: int, cols: int, row_stride: int, tokens: int | None,
                     token_stride: int, width: int, lengths: int | None, prompts: int | None, repetition: int | None,
                     presence: int | None, frequency: int | None, bias_token: int | None, bias_value: int | None,
                     bias_stride: int, biases: int, allowed: int | None, allowed_stride: int, out: int,
                     out_stride: int, stream: int | None) -> int:
    """The C entry point of penalties, biases and masks with raw pointers; returns the status code."""
    return library().tf_topk_penalize(logits, dtype, rows, cols, row_stride, tokens, token_stride, width, lengths,
                                      prompts, repetition, presence, frequency, bias_token, bias_value, bias_stride,
                                      biases, allowed, allowed_stride, out, out_stride, stream)


def _per_row(t, rows, dtype, dev, name):
    """Address of an optional [rows] tensor, checked."""
    if t is None:
        return None
    _check_out(t, (rows,), dtype, dev, name)
    return t.data_ptr()


def _table(t, rows, dtype, dev, name):
    """(address, width, row stride) of an optional [rows, width] tensor with contiguous columns, checked."""
    if t is None:
        return None, 0, 0
    if t.dtype is not dtype or t.device != dev or t.dim() != 2 or t.shape[0] != rows:
        raise ValueError(f"{name} must be a 2-D {dtype} tensor with the logits' rows, on their device")
    width, stride = t.shape[1], t.stride()
    if width > 1 and stride[1] != 1:
        raise ValueError(f"{name} must have contiguous columns")
    if width > _INT32_MAX:
        _check(ERR_SHAPE)
    return t.data_ptr(), width, stride[0] if rows > 1 else width


def penalize_logits(logits, *, tokens=None, lengths=None, prompts=None, repetition=None, presence=None, frequency=None,
                    bias_tokens=None, bias_values=None, allowed=None, out=None, stream=None):
    """Logits made ready for ``select_topk``: penalties for each request's
    tokens so far, biases and a grammar's mask, in one pass.

    ``logits``: CUDA bf16 / fp16 / fp32 [rows, cols], contiguous columns.
    ``tokens``: int32 [rows, width]; row r's first ``prompts[r]`` (int32; none
    if None) are its prompt, those up to ``lengths[r]`` (int32; all if None)
    its answer so far.  ``repetition`` (over prompt and answer: a positive
    logit is divided by it, any other multiplied), ``presence`` and
    ``frequency`` (over the answer: subtracted once, and once for each time):
    float32 [rows].  ``bias_tokens`` int32 and ``bias_values`` float32 [rows,
    biases]: added to those columns (of several entries for one column the
    last counts; columns out of range are passed over).  ``allowed``: int32
    [rows, ceil(cols / 32)], bit c % 32 of word c // 32 set where column c
    stays; the others become -inf.
    Returns [rows, cols] of the logits' dtype; ``out`` may be ``logits`` itself.
    """
    code, rows, cols, stride = _rows_code(logits, "logits")
    torch, dev = _torch, logits.device
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return penalize_logits(logits, tokens=tokens, lengths=lengths, prompts=prompts, repetition=repetition,
                                   presence=presence, frequency=frequency, bias_tokens=bias_tokens,
                                   bias_values=bias_values, allowed=allowed, out=out, stream=stream)
    said, width, said_stride = _table(tokens, rows, torch.int32, dev, "tokens")
    names, biases, bias_stride = _table(bias_tokens, rows, torch.int32, dev, "bias_tokens")
    values, count, value_stride = _table(bias_values, rows, torch.float32, dev, "bias_values")
    if count != biases or value_stride != bias_stride:
        raise ValueError("bias_tokens and bias_values must have one shape and one row stride")
    mask, words, mask_stride = _table(allowed, rows, torch.int32, dev, "allowed")
    if allowed is not None and words != -(-cols // 32):
        raise ValueError("allowed must have a bit for each column, in words of 32")
    if out is None:
        out, out_stride = _empty((rows, cols), logits.dtype, dev, stream), cols
    elif out is logits:
        out_stride = stride
    else:
        if out.dtype is not logits.dtype or out.device != dev or tuple(out.shape) != (rows, cols):
            raise ValueError("out must have the logits' shape, dtype and device")
        out_stride = _rows_code(out, "out")[3]
    _check((_lib or library()).tf_topk_penalize(
        logits.data_ptr(), code, rows, cols, stride, said, said_stride, width,
        _per_row(lengths, rows, torch.int32, dev, "lengths"), _per_row(prompts, rows, torch.int32, dev, "prompts"),
        _per_row(repetition, rows, torch.float32, dev, "repetition"),
        _per_row(presence, rows, torch.float32, dev, "presence"),
        _per_row(frequency, rows, torch.float32, dev, "frequency"), names, values, bias_stride, biases, mask,
        mask_stride, out.data_ptr(), out_stride, _stream_handle(stream, dev)))
    return out


def device_fault() -> int:
    """0, or the fault code a kernel recorded since the last check (then cleared)."""
    r = library().tf_topk_device_fault()
    if r < 0:
        _check(-r)
    return r


def plan(rows: int, cols: int, k: int) -> int:
    """Launch plan (TF_TOPK_PLAN_* code) the library picks for a shape on the current device."""
    r = library().tf_topk_bf16_plan(rows, cols, k)
    if r < 0:
        _check(-r)
    return r


def topk_bf16(x, k: int, *, plan: int = 0, out=None, stream=None):
    """Exact top-k of every row of a CUDA bf16 matrix.

    ``x``: a CUDA tensor of dtype bfloat16 (or int16/uint16 holding bf16 bits),
    1-D (one row) or 2-D with unit column stride; ``x.stride(0)`` is the row
    stride, so a column-sliced view of a padded buffer works as is.
    Returns ``(idx int32[rows,k], val bfloat16[rows,k], count int32[rows],
    mask int32[rows])``; ``mask`` holds the uint32 bits (1 NaN, 2 +inf, 4 -inf).
    ``out`` may supply those four tensors.  Runs on ``stream`` (a
    ``torch.cuda.Stream``) or the current stream of ``x``'s device.  ``plan``
    picks the launch plan (``PLANS``; 0 = the library's choice); every plan
    gives the same result.
    """
    import torch

    if not x.is_cuda:
        raise ValueError("topk_bf16 needs a CUDA tensor (no CPU path exists)")
    if x.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"expected bf16 bits, got {x.dtype}")
    if x.dim() == 1:
        x = x.unsqueeze(0)
    if x.dim() != 2:
        raise ValueError("x must be 1-D or 2-D")
    rows, cols = x.shape
    if cols > 1 and x.stride(1) != 1:
        raise ValueError("columns must be contiguous (stride(1) == 1)")
    row_stride = x.stride(0) if rows > 1 else max(cols, x.stride(0))
    dev = x.device
    if out is None:
        idx = torch.empty((rows, k), dtype=torch.int32, device=dev)
        val = torch.empty((rows, k), dtype=torch.bfloat16, device=dev)
        count = torch.empty((rows,), dtype=torch.int32, device=dev)
        mask = torch.empty((rows,), dtype=torch.int32, device=dev)
    else:
        idx, val, count, mask = out
        for t, shape, dtypes in ((idx, (rows, k), (torch.int32,)),
                                 (val, (rows, k), (torch.bfloat16, torch.int16, torch.uint16)),
                                 (count, (rows,), (torch.int32,)),
                                 (mask, (rows,), (torch.int32, torch.uint32))):
            if tuple(t.shape) != shape or t.dtype not in dtypes or not t.is_contiguous() \
                    or t.device != dev:
                raise ValueError("out tensors must be contiguous, on x's device, with shapes "
                                 "(rows,k), (rows,k), (rows,), (rows,)")
    _check(_on_device(dev, library().tf_topk_bf16_with_plan, x.data_ptr(), rows, cols, row_stride, k,
                      idx.data_ptr(), val.data_ptr(), count.data_ptr(), mask.data_ptr(), plan,
                      _stream_handle(stream, dev)))
    return idx, val, count, mask
