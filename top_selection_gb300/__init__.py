"""GB300-native DeepSelect row-wise top-k.

A thin ctypes binding over ``libds_topk.so`` (built in-tree from ``csrc/`` by
``top_selection_gb300.build``).  Functions carry the C ABI's names and do argument
marshalling only: every step of the computation runs in the library's CUDA kernels.
There is no CPU fallback; when the library has not been built every call raises.

The C ABI (``include/ds_topk.h``) documents the operation, the argument layout, the
ownership rules and the error codes.  ``topk()`` is a convenience wrapper that takes and
returns torch tensors (PyTorch supplies device memory and streams only).

The operators around the top-k in a decoding step -- ``route``, ``route_backward``,
``verify_drafts``, ``cache_store``, ``cache_load``, ``cache_attention`` -- and what follows the
selections -- ``token_logprobs`` and ``token_logprobs_backward``; ``expert_sort``, ``expert_gather``,
``expert_combine`` and ``expert_combine_backward``; ``quantise_blocks`` and ``expert_product`` -- take and
return torch tensors as well; their checks, outputs and calls run in a compiled binding
(``csrc/ds_torch.cpp``), since a step makes many small ones.  They run on their tensors' device, on
its current stream or on ``stream`` (a raw handle): then inputs have to be ready there and stay until
the call's work is done, and outputs come from that stream's memory.
"""
from __future__ import annotations

import ctypes
import importlib
import os
import threading

__all__ = [
    "DS_BF16", "DS_FP32", "DS_NSTAT", "DSError", "ds_topk", "ds_topk_ex", "ds_get_plan",
    "ds_workspace_bytes", "ds_get_device_status", "ds_status_string", "ds_version",
    "ds_block_order", "ds_wait_probe", "ds_topk_noalloc", "ds_noalloc_scratch_bytes", "topk",
    "library_path", "load",
    "DS_SOFTMAX", "DS_SIGMOID", "DS_GROUP_MAX", "DS_GROUP_TOP2", "ds_topk_sample", "topk_sample",
    "ds_route", "ds_route_backward", "ds_verify_drafts", "ds_cache_store", "ds_cache_load", "ds_cache_attention",
    "ds_cache_attention_ex", "ds_cache_attention_workspace_bytes",
    "route", "route_backward", "verify_drafts", "cache_store", "cache_load", "cache_attention",
    "ds_token_logprobs", "ds_token_logprobs_backward", "ds_expert_sort", "ds_expert_gather", "ds_expert_combine",
    "ds_expert_combine_backward", "ds_quantise_blocks", "ds_expert_gather_quantised", "ds_expert_product",
    "ds_expert_product_probe",
    "token_logprobs", "token_logprobs_backward", "expert_sort", "expert_gather", "expert_combine",
    "expert_combine_backward", "quantise_blocks", "expert_product",
]

DS_BF16 = 0
DS_FP32 = 1
DS_NSTAT = 8
DS_SOFTMAX = 0
DS_SIGMOID = 1
DS_GROUP_MAX = 0
DS_GROUP_TOP2 = 1

STATUS_NAMES = {
    0: "DS_OK", 1: "DS_ERR_INVALID_ARG", 2: "DS_ERR_ALIGNMENT", 3: "DS_ERR_UNSUPPORTED",
    4: "DS_ERR_CUDA", 5: "DS_ERR_TIMEOUT", 6: "DS_ERR_INTERNAL", 7: "DS_ERR_WORKSPACE",
}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libds_topk.so")
_lock = threading.Lock()
_lib = None


class DSError(RuntimeError):
    def __init__(self, status: int, what: str = "ds_topk"):
        self.status = int(status)
        super().__init__(f"{what} failed: {STATUS_NAMES.get(self.status, self.status)} "
                         f"({ds_status_string(self.status) if _lib else ''})")


class ds_options(ctypes.Structure):
    _fields_ = [("parts", ctypes.c_int32), ("cluster", ctypes.c_int32),
                ("stats", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("input_ready", ctypes.c_int32),
                ("sorted", ctypes.c_int32)]


class ds_plan(ctypes.Structure):
    _fields_ = [("parts", ctypes.c_int32), ("cluster", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("chunk_elems", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("capacity", ctypes.c_int32),
                ("smem_bytes", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
                ("ctas_per_sm", ctypes.c_int32), ("merge_launch", ctypes.c_int32),
                ("B", ctypes.c_int32), ("B2", ctypes.c_int32), ("spec_k", ctypes.c_int32)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libds_topk.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                               "`python -m top_selection_gb300.build` (nvcc, sm_103a)")
        lib = ctypes.CDLL(_LIB_PATH)
        i32, i64, u64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_size_t
        lib.ds_topk.argtypes = [vp, i32, i64, i64, i64, i32, i32, i32, u64, vp, vp, vp]
        lib.ds_topk.restype = ctypes.c_int
        lib.ds_topk_ex.argtypes = [vp, i32, i64, i64, i64, i32, i32, i32, u64, vp, vp,
                                   ctypes.POINTER(ds_options), vp]
        lib.ds_topk_ex.restype = ctypes.c_int
        lib.ds_get_plan.argtypes = [i32, i64, i64, i32, i32, i32, ctypes.POINTER(ds_options),
                                    ctypes.POINTER(ds_plan)]
        lib.ds_get_plan.restype = ctypes.c_int
        lib.ds_workspace_bytes.argtypes = [i32, i64, i64, i32, i32, i32, ctypes.POINTER(ds_options),
                                           ctypes.POINTER(sz)]
        lib.ds_workspace_bytes.restype = ctypes.c_int
        lib.ds_get_device_status.argtypes = [vp]
        lib.ds_get_device_status.restype = ctypes.c_int
        lib.ds_status_string.argtypes = [ctypes.c_int]
        lib.ds_status_string.restype = ctypes.c_char_p
        lib.ds_version.argtypes = []
        lib.ds_version.restype = ctypes.c_char_p
        lib.ds_block_order.argtypes = [u64, i64, i64, i32, vp, vp]
        lib.ds_block_order.restype = ctypes.c_int
        lib.ds_wait_probe.argtypes = [i64, vp]
        lib.ds_wait_probe.restype = ctypes.c_int
        lib.ds_topk_noalloc.argtypes = [vp, i32, i64, i64, i64, i32, i32, i32, u64, vp, vp, i32, i32, vp]
        lib.ds_topk_noalloc.restype = ctypes.c_int
        lib.ds_topk_sample.argtypes = [vp, i32, i64, i64, i64, i32, i32, i32, u64, ctypes.c_float, vp, vp, vp,
                                       vp, vp, vp]
        lib.ds_topk_sample.restype = ctypes.c_int
        lib.ds_noalloc_scratch_bytes.argtypes = []
        lib.ds_noalloc_scratch_bytes.restype = ctypes.c_size_t
        f32 = ctypes.c_float
        lib.ds_route.argtypes = [vp, i32, i64, i32, i64, i32, i32, vp, i32, i32, i32, i32, f32, vp, vp, vp, vp]
        lib.ds_route.restype = ctypes.c_int
        lib.ds_route_backward.argtypes = [vp, vp, i32, i64, i32, i64, i32, vp, i32, i32, f32, vp, i64, vp]
        lib.ds_route_backward.restype = ctypes.c_int
        lib.ds_verify_drafts.argtypes = [vp, i32, i64, i32, i64, i64, i64, vp, vp, vp, i64, i64, vp, vp, i64, vp, f32,
                                         vp, vp, vp, vp]
        lib.ds_verify_drafts.restype = ctypes.c_int
        lib.ds_cache_store.argtypes = [vp, vp, i32, i64, i32, i32, i64, i64, i64, i64, vp, vp, i64, i32, vp, vp]
        lib.ds_cache_store.restype = ctypes.c_int
        lib.ds_cache_load.argtypes = [vp, vp, i64, i32, vp, i64, i32, i32, i32, vp, vp, vp]
        lib.ds_cache_load.restype = ctypes.c_int
        lib.ds_cache_attention.argtypes = [vp, i32, i64, i32, i32, i32, i64, i64, i64, vp, vp, i64, i32, i32, vp, i64,
                                           i64, vp, vp, i32, f32, vp, vp, vp]
        lib.ds_cache_attention.restype = ctypes.c_int
        lib.ds_cache_attention_ex.argtypes = [*lib.ds_cache_attention.argtypes[:-1], vp, ctypes.c_size_t, vp]
        lib.ds_cache_attention_ex.restype = ctypes.c_int
        lib.ds_cache_attention_workspace_bytes.argtypes = [i32, i64, i32, i32, i32, i32, i32, i64, i32, i32,
                                                           ctypes.POINTER(ctypes.c_size_t)]
        lib.ds_cache_attention_workspace_bytes.restype = ctypes.c_int
        lib.ds_token_logprobs.argtypes = [vp, i32, i64, i64, i64, vp, i32, vp, vp, vp, vp, vp, vp]
        lib.ds_token_logprobs.restype = ctypes.c_int
        lib.ds_token_logprobs_backward.argtypes = [vp, vp, i32, i64, i64, i64, vp, vp, vp, vp, vp, i64, vp]
        lib.ds_token_logprobs_backward.restype = ctypes.c_int
        lib.ds_expert_sort.argtypes = [vp, i64, i32, i32, vp, vp, vp]
        lib.ds_expert_sort.restype = ctypes.c_int
        lib.ds_expert_gather.argtypes = [vp, i32, i64, i32, i64, vp, i32, vp, i32, vp, vp]
        lib.ds_expert_gather.restype = ctypes.c_int
        lib.ds_expert_combine.argtypes = [vp, i32, i64, i32, i64, vp, i64, i32, vp, vp, vp]
        lib.ds_expert_combine.restype = ctypes.c_int
        lib.ds_expert_combine_backward.argtypes = [vp, i64, vp, i32, i32, i64, vp, i64, i32, vp, i32, vp, vp, vp, vp]
        lib.ds_expert_combine_backward.restype = ctypes.c_int
        lib.ds_quantise_blocks.argtypes = [vp, i32, i64, i64, i32, i64, i64, i32, vp, vp, vp]
        lib.ds_quantise_blocks.restype = ctypes.c_int
        lib.ds_expert_gather_quantised.argtypes = [vp, i32, i64, i32, i64, vp, i32, vp, i32, vp, vp, vp]
        lib.ds_expert_gather_quantised.restype = ctypes.c_int
        lib.ds_expert_product.argtypes = [vp, vp, i64, i32, i64, vp, vp, i32, i32, i64, i64, vp, i32, vp, vp]
        lib.ds_expert_product.restype = ctypes.c_int
        lib.ds_expert_product_probe.argtypes = [i32] + lib.ds_expert_product.argtypes
        lib.ds_expert_product_probe.restype = ctypes.c_int
        _lib = lib
        return lib


def _opts(parts=0, cluster=0, stats=0, workspace=0, workspace_bytes=0, input_ready=False, sorted=False):
    return ds_options(int(parts), int(cluster), int(stats) or None, int(workspace) or None,
                      int(workspace_bytes), 1 if input_ready else 0, 1 if sorted else 0)


# ------------------------------------------------------------------ C ABI mirror ----

def ds_topk(x, dtype, rows, N, row_stride, k, B, B2, seed, out_vals, out_idx, stream=0) -> int:
    """Raw C call with device pointers (ints); returns the ds_status code."""
    return load().ds_topk(int(x) or None, dtype, rows, N, row_stride, k, B, B2, seed,
                          int(out_vals) or None, int(out_idx) or None, int(stream) or None)


def ds_topk_ex(x, dtype, rows, N, row_stride, k, B, B2, seed, out_vals, out_idx,
               parts=0, cluster=0, stats=0, workspace=0, workspace_bytes=0, input_ready=False,
               stream=0, sorted=False) -> int:
    o = _opts(parts, cluster, stats, workspace, workspace_bytes, input_ready, sorted)
    return load().ds_topk_ex(int(x) or None, dtype, rows, N, row_stride, k, B, B2, seed,
                             int(out_vals) or None, int(out_idx) or None, ctypes.byref(o),
                             int(stream) or None)


def ds_get_plan(dtype, rows, N, k, B, B2, parts=0, cluster=0, stats=False) -> dict:
    o = _opts(parts, cluster, 1 if stats else 0)
    p = ds_plan()
    st = load().ds_get_plan(dtype, rows, N, k, B, B2, ctypes.byref(o), ctypes.byref(p))
    if st != 0:
        raise DSError(st, "ds_get_plan")
    return p.as_dict()


def ds_workspace_bytes(dtype, rows, N, k, B, B2, parts=0, cluster=0) -> int:
    o = _opts(parts, cluster)
    out = ctypes.c_size_t(0)
    st = load().ds_workspace_bytes(dtype, rows, N, k, B, B2, ctypes.byref(o), ctypes.byref(out))
    if st != 0:
        raise DSError(st, "ds_workspace_bytes")
    return int(out.value)


def ds_get_device_status(stream=0) -> int:
    return load().ds_get_device_status(int(stream) or None)


def ds_status_string(status: int) -> str:
    return load().ds_status_string(int(status)).decode()


def ds_version() -> str:
    return load().ds_version().decode()


def ds_block_order(seed, row, first_block, nblocks, out_perm, stream=0) -> int:
    return load().ds_block_order(seed, row, first_block, nblocks, int(out_perm), int(stream) or None)


def ds_wait_probe(cycles, stream=0) -> int:
    return load().ds_wait_probe(int(cycles), int(stream) or None)


def ds_topk_noalloc(x, dtype, rows, N, row_stride, k, B, B2, seed, out_vals, out_idx, parts=0, cluster=0,
                    stream=0) -> int:
    """ds_topk for callers that cannot allocate: scratch comes from a fixed array in the
    library (see include/ds_topk.h).  Raw device pointers; returns the ds_status code."""
    return load().ds_topk_noalloc(int(x) or None, dtype, rows, N, row_stride, k, B, B2, seed,
                                  int(out_vals) or None, int(out_idx) or None, parts, cluster,
                                  int(stream) or None)


def ds_noalloc_scratch_bytes() -> int:
    return int(load().ds_noalloc_scratch_bytes())


# ------------------------------------------------------------------ torch helper ----

def _torch_dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16 or t.dtype in (torch.int16, torch.uint16):
        return DS_BF16
    if t.dtype in (torch.float32, torch.int32):
        return DS_FP32
    raise TypeError(f"unsupported dtype {t.dtype}: bf16 (or 16-bit patterns) and fp32 only")


def topk(x, k: int, B: int, B2: int, seed: int = 0x5EED, N: int | None = None,
         out=None, parts: int = 0, cluster: int = 0, stats=None, workspace=None, stream=None,
         input_ready: bool = False, sorted: bool = False):
    """Row-wise DeepSelect top-k of a CUDA tensor ``x`` of shape (rows, stride).

    Returns (values, indices), each (rows, k), unordered within a row unless ``sorted``
    (then by value descending, equal values by column ascending).  ``N`` (default:
    the row length) may be shorter than the stride.  ``stats`` is an optional int64
    CUDA tensor (rows, DS_NSTAT) filled when each row is one part.  ``input_ready`` states
    that ``x`` was complete before the previous kernel on the stream started, which lets
    the call start reading it while that kernel finishes."""
    import torch
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor (there is no CPU path)")
    if x.dim() == 1:
        x = x.view(1, -1)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    dtype = _torch_dtype_code(x)
    rows = x.shape[0]
    n = x.shape[1] if N is None else int(N)
    stride = x.stride(0) if rows > 1 else x.shape[1]
    if out is None:
        vals = torch.empty((rows, k), dtype=x.dtype, device=x.device)
        idx = torch.empty((rows, k), dtype=torch.int32, device=x.device)
    else:
        vals, idx = out
    if stream is None:
        stream = torch.cuda.current_stream(x.device).cuda_stream
    ws_ptr, ws_bytes = 0, 0
    if workspace is not None:
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = ds_topk_ex(x.data_ptr(), dtype, rows, n, stride, k, B, B2, seed, vals.data_ptr(),
                    idx.data_ptr(), parts=parts, cluster=cluster,
                    stats=0 if stats is None else stats.data_ptr(), workspace=ws_ptr,
                    workspace_bytes=ws_bytes, input_ready=input_ready, stream=stream, sorted=sorted)
    if st != 0:
        raise DSError(st)
    return vals, idx


def ds_topk_sample(x, dtype, rows, N, row_stride, k, B, B2, seed, temperature, uniforms, out_vals, out_idx,
                   out_token, out_prob=0, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_topk_sample(int(x) or None, dtype, rows, N, row_stride, k, B, B2, seed, float(temperature),
                                 int(uniforms) or None, int(out_vals) or None, int(out_idx) or None,
                                 int(out_token) or None, int(out_prob) or None, int(stream) or None)


def topk_sample(x, k: int, temperature: float, uniforms, B: int = 0, B2: int = 0, seed: int = 0x5EED,
                N: int | None = None, stream=None):
    """Top-k sampling of each row of the CUDA logits tensor ``x`` (rows, stride): the
    sorted top-k (values, columns), then one column drawn per row from the softmax of the
    k values at ``temperature`` with the row's uniform draw from ``uniforms`` (a CUDA
    float32 tensor of rows values in [0, 1)).  Returns (token, prob, values, indices)."""
    import torch
    if not x.is_cuda or not uniforms.is_cuda:
        raise ValueError("x and uniforms must be CUDA tensors (there is no CPU path)")
    if x.dim() == 1:
        x = x.view(1, -1)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    if uniforms.dtype != torch.float32 or uniforms.numel() != x.shape[0] or not uniforms.is_contiguous():
        raise ValueError("uniforms must be a contiguous float32 tensor with one value per row")
    dtype = _torch_dtype_code(x)
    rows = x.shape[0]
    n = x.shape[1] if N is None else int(N)
    stride = x.stride(0) if rows > 1 else x.shape[1]
    vals = torch.empty((rows, k), dtype=x.dtype, device=x.device)
    idx = torch.empty((rows, k), dtype=torch.int32, device=x.device)
    token = torch.empty(rows, dtype=torch.int32, device=x.device)
    prob = torch.empty(rows, dtype=torch.float32, device=x.device)
    if stream is None:
        stream = torch.cuda.current_stream(x.device).cuda_stream
    st = ds_topk_sample(x.data_ptr(), dtype, rows, n, stride, k, B, B2, seed, temperature, uniforms.data_ptr(),
                        vals.data_ptr(), idx.data_ptr(), token.data_ptr(), prob.data_ptr(), stream)
    if st != 0:
        raise DSError(st, "ds_topk_sample")
    return token, prob, vals, idx


# --------------------------------------------- operators around the top-k ----------

def ds_route(logits, dtype, rows, E, row_stride, k, scoring, bias, groups, topk_groups, group_score, renormalise,
             scale, out_weights, out_experts, counts=0, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_route(int(logits) or None, dtype, rows, E, row_stride, k, scoring, int(bias) or None, groups,
                           topk_groups, group_score, int(bool(renormalise)), float(scale), int(out_weights) or None,
                           int(out_experts) or None, int(counts) or None, int(stream) or None)


def ds_route_backward(grad_weights, logits, dtype, rows, E, row_stride, k, experts, scoring, renormalise, scale,
                      grad_logits, grad_stride, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_route_backward(int(grad_weights) or None, int(logits) or None, dtype, rows, E, row_stride, k,
                                    int(experts) or None, scoring, int(bool(renormalise)), float(scale),
                                    int(grad_logits) or None, grad_stride, int(stream) or None)


def ds_verify_drafts(logits, dtype, sequences, drafts_per_sequence, V, seq_stride, row_stride, drafts, draft_lens,
                     draft_probs, probs_seq_stride, probs_row_stride, uniforms, noise, noise_stride, temperatures,
                     temperature, out_tokens, out_accepted, out_probs=0, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_verify_drafts(int(logits) or None, dtype, sequences, drafts_per_sequence, V, seq_stride,
                                   row_stride, int(drafts) or None, int(draft_lens) or None, int(draft_probs) or None,
                                   probs_seq_stride, probs_row_stride, int(uniforms) or None, int(noise) or None,
                                   noise_stride, int(temperatures) or None, float(temperature),
                                   int(out_tokens) or None, int(out_accepted) or None, int(out_probs) or None,
                                   int(stream) or None)


def ds_cache_store(k, v, dtype, tokens, heads, D, k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                   cache, scales, pages, page, slots, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_cache_store(int(k) or None, int(v) or None, dtype, tokens, heads, D, k_token_stride,
                                 k_head_stride, v_token_stride, v_head_stride, int(cache) or None,
                                 int(scales) or None, pages, page, int(slots) or None, int(stream) or None)


def ds_cache_load(cache, scales, pages, page, slots, tokens, heads, D, dtype, out_k, out_v, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_cache_load(int(cache) or None, int(scales) or None, pages, page, int(slots) or None, tokens,
                                heads, D, dtype, int(out_k) or None, int(out_v) or None, int(stream) or None)


def ds_cache_attention(q, dtype, sequences, tokens, q_heads, D, q_seq_stride, q_token_stride, q_head_stride, cache,
                       scales, pages, heads, page, table, table_width, table_stride, lens, indices, K, scale, out,
                       out_lse=0, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_cache_attention(int(q) or None, dtype, sequences, tokens, q_heads, D, q_seq_stride,
                                     q_token_stride, q_head_stride, int(cache) or None, int(scales) or None, pages,
                                     heads, page, int(table) or None, table_width, table_stride, int(lens) or None,
                                     int(indices) or None, K, float(scale), int(out) or None, int(out_lse) or None,
                                     int(stream) or None)


def ds_cache_attention_ex(q, dtype, sequences, tokens, q_heads, D, q_seq_stride, q_token_stride, q_head_stride, cache,
                          scales, pages, heads, page, table, table_width, table_stride, lens, indices, K, scale, out,
                          out_lse=0, workspace=0, workspace_bytes=0, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_cache_attention_ex(int(q) or None, dtype, sequences, tokens, q_heads, D, q_seq_stride,
                                        q_token_stride, q_head_stride, int(cache) or None, int(scales) or None, pages,
                                        heads, page, int(table) or None, table_width, table_stride, int(lens) or None,
                                        int(indices) or None, K, float(scale), int(out) or None, int(out_lse) or None,
                                        int(workspace) or None, workspace_bytes, int(stream) or None)


def ds_cache_attention_workspace_bytes(dtype, sequences, tokens, q_heads, D, heads, page, table_width, picked=False,
                                       K=0) -> int:
    out = ctypes.c_size_t(0)
    st = load().ds_cache_attention_workspace_bytes(dtype, sequences, tokens, q_heads, D, heads, page, table_width,
                                                   int(bool(picked)), K, ctypes.byref(out))
    if st != 0:
        raise DSError(st, "ds_cache_attention_workspace_bytes")
    return int(out.value)


def ds_token_logprobs(logits, dtype, rows, V, row_stride, tokens, top, out_logprobs, out_lse, out_entropy,
                      out_top_logprobs=0, out_top_tokens=0, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_token_logprobs(int(logits) or None, dtype, rows, V, row_stride, int(tokens) or None, top,
                                    int(out_logprobs) or None, int(out_lse) or None, int(out_entropy) or None,
                                    int(out_top_logprobs) or None, int(out_top_tokens) or None, int(stream) or None)


def ds_token_logprobs_backward(grad_logprobs, logits, dtype, rows, V, row_stride, tokens, lse, grad_entropy, entropy,
                               grad_logits, grad_stride, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_token_logprobs_backward(int(grad_logprobs) or None, int(logits) or None, dtype, rows, V, row_stride,
                                             int(tokens) or None, int(lse) or None, int(grad_entropy) or None,
                                             int(entropy) or None, int(grad_logits) or None, grad_stride,
                                             int(stream) or None)


def ds_expert_sort(experts, tokens, k, E, places, offsets, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_expert_sort(int(experts) or None, tokens, k, E, int(places) or None, int(offsets) or None,
                                 int(stream) or None)


def ds_expert_gather(x, dtype, tokens, D, row_stride, places, k, offsets, E, out, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_expert_gather(int(x) or None, dtype, tokens, D, row_stride, int(places) or None, k,
                                   int(offsets) or None, E, int(out) or None, int(stream) or None)


def ds_expert_combine(y, dtype, rows, D, row_stride, places, tokens, k, weights, out, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_expert_combine(int(y) or None, dtype, rows, D, row_stride, int(places) or None, tokens, k,
                                    int(weights) or None, int(out) or None, int(stream) or None)


def ds_expert_combine_backward(grad, grad_stride, y, dtype, D, row_stride, places, tokens, k, offsets, E, weights,
                               grad_y, grad_weights, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_expert_combine_backward(int(grad) or None, grad_stride, int(y) or None, dtype, D, row_stride,
                                             int(places) or None, tokens, k, int(offsets) or None, E,
                                             int(weights) or None, int(grad_y) or None, int(grad_weights) or None,
                                             int(stream) or None)


def ds_quantise_blocks(x, dtype, matrices, rows, K, matrix_stride, row_stride, block_rows, codes, scales,
                       stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_quantise_blocks(int(x) or None, dtype, matrices, rows, K, matrix_stride, row_stride, block_rows,
                                     int(codes) or None, int(scales) or None, int(stream) or None)


def ds_expert_gather_quantised(x, dtype, tokens, D, row_stride, places, k, offsets, E, codes, scales, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_expert_gather_quantised(int(x) or None, dtype, tokens, D, row_stride, int(places) or None, k,
                                             int(offsets) or None, E, int(codes) or None, int(scales) or None,
                                             int(stream) or None)


def ds_expert_product(x, x_scales, rows, K, x_stride, w, w_scales, E, N, w_row_stride, w_matrix_stride, offsets, dtype,
                      out, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_expert_product(int(x) or None, int(x_scales) or None, rows, K, x_stride, int(w) or None,
                                    int(w_scales) or None, E, N, w_row_stride, w_matrix_stride, int(offsets) or None,
                                    dtype, int(out) or None, int(stream) or None)


def ds_expert_product_probe(block, x, x_scales, rows, K, x_stride, w, w_scales, E, N, w_row_stride, w_matrix_stride,
                            offsets, dtype, out, stream=0) -> int:
    """Raw C call (device pointers as ints); returns the ds_status code."""
    return load().ds_expert_product_probe(block, int(x) or None, int(x_scales) or None, rows, K, x_stride, int(w) or None,
                                          int(w_scales) or None, E, N, w_row_stride, w_matrix_stride, int(offsets) or None,
                                          dtype, int(out) or None, int(stream) or None)


class _Names(dict):
    """Values by name; a name that is none of them is refused."""

    def __missing__(self, name):
        raise ValueError(f"{name!r} is none of {sorted(map(str, self))}")


_SCORING = _Names(softmax=DS_SOFTMAX, sigmoid=DS_SIGMOID)
_GROUP_SCORE = _Names(max=DS_GROUP_MAX, top2=DS_GROUP_TOP2)
_binding = None         # the compiled tensor binding (csrc/ds_torch.cpp), loaded on first use


def _load_binding():
    """Loads the tensor binding: it checks tensors, allocates outputs and calls the C ABI."""
    global _binding
    load()
    with _lock:
        if _binding is None:
            import torch  # noqa: F401  (the binding's own libraries)
            from . import build
            missing = ("the tensor binding is missing or was built for another torch: build it with "
                       "`python -m top_selection_gb300.build`")
            if not build.binding_matches():
                raise RuntimeError(missing)
            try:
                ops = importlib.import_module("._ops", __name__)
            except ImportError as e:
                raise RuntimeError(missing) from e
            ops.set_error(DSError)
            _binding = ops
    return _binding


def route(logits, k: int, scoring: str = "softmax", bias=None, groups: int = 1, topk_groups: int = 1,
          group_score: str = "max", renormalise: bool = True, scale: float = 1.0, counts=None, stream=None):
    """The experts' gate: each row's k best experts of ``logits`` (rows, E) and their weights.

    Scores are a softmax or a logistic function of the logits; ``bias`` (E,) is added for the
    choice only; with ``groups`` > 1 only experts of the ``topk_groups`` best groups are
    eligible (a group's score: "max", or "top2", the sum of its two largest).  Weights are
    ``scale`` times the scores, divided by their sum over the chosen with ``renormalise``.
    ``counts`` (E,) int32, if given, is added the number of rows that chose each expert.
    Returns (weights (rows, k) float32, experts (rows, k) int32), best first, ties to the lower
    index.  The weights carry no autograd history: ``route_backward`` gives their gradient."""
    return (_binding or _load_binding()).route(logits, k, _SCORING[scoring], bias, groups, topk_groups,
                                                 _GROUP_SCORE[group_score], renormalise, scale, counts, stream)


def route_backward(grad_weights, logits, experts, scoring: str = "softmax", renormalise: bool = True,
                   scale: float = 1.0, stream=None):
    """The gradient of ``route``'s weights with respect to its ``logits`` (rows, E), for the
    ``experts`` it chose: (rows, E) in the logits' dtype.  Other arguments as in ``route``."""
    return (_binding or _load_binding()).route_backward(grad_weights, logits, experts, _SCORING[scoring], renormalise, scale,
                                                          stream)


def verify_drafts(logits, drafts, uniforms, noise, draft_probs=None, draft_lens=None, temperature=1.0, stream=None):
    """Verifies each sequence's drafted tokens against the target's ``logits`` (B, S + 1, V) and
    emits one more token: speculative sampling with the caller's random numbers.

    ``drafts`` (B, S) int32, drawn from ``draft_probs`` (B, S, V) float32 (None: looked-up
    drafts, one-hot); ``draft_lens`` (B,) int32 drafts of each sequence (None: S);
    ``uniforms`` (B, S) in [0, 1); ``noise`` (B, V) exponential draws; ``temperature`` a number or
    a (B,) float32 tensor, 0 for the likeliest token.  Returns (tokens (B, S + 1) int32 -- the
    accepted drafts, the emitted token, then -1 -- accepted (B,) int32, and the target's
    probability of each token (B, S + 1) float32)."""
    return (_binding or _load_binding()).verify_drafts(logits, drafts, uniforms, noise, draft_probs, draft_lens,
                                                         temperature, stream)


def cache_store(k, v, cache, scales, slots, stream=None) -> None:
    """Writes keys and values ``k``, ``v`` (tokens, heads, D) to the ``slots`` (tokens,) int32 of a
    4-bit cache: ``cache`` (pages, heads, page, 2, D / 2) uint8 and ``scales`` (pages, heads, page,
    4) bfloat16.  Slot t is place t % page of page t / page; a negative slot is skipped."""
    (_binding or _load_binding()).cache_store(k, v, cache, scales, slots, stream)


def cache_load(cache, scales, slots, dtype=None, stream=None):
    """Reads the ``slots`` (tokens,) int32 of a 4-bit cache back: keys and values (tokens, heads,
    D) in ``dtype`` (bfloat16, the default, or float32); zeros for a slot outside the cache."""
    ops = _binding or _load_binding()
    if dtype is not None and str(dtype) not in ("torch.bfloat16", "torch.float32"):
        raise TypeError(f"dtype: unsupported dtype {dtype}: bfloat16 and float32 only")
    return ops.cache_load(cache, scales, slots, str(dtype) == "torch.float32", stream)


def cache_attention(q, cache, scales, table, lens, indices=None, scale=None, stream=None):
    """Attention of each sequence's newest tokens ``q`` (B, Q, query heads, D) over a 4-bit cache.

    ``table`` (B, width) int32 holds the page of each run of ``page`` positions, ``lens`` (B,) int32
    the positions stored, the Q new ones among them: token i sees those below lens - (Q - 1 - i),
    or those of them that ``indices`` (B, Q, K) int32 lists (``topk``'s columns; -1 pads).  ``scale``
    is 1 / sqrt(D) by default.  Returns (out (B, Q, query heads, D) in q's dtype, lse (B, Q, query
    heads) float32); a token that sees nothing gives 0 and -inf."""
    return (_binding or _load_binding()).cache_attention(q, cache, scales, table, lens, indices, scale, stream)


# --------------------------------------------- behind the selections ----------------

def token_logprobs(logits, tokens, top: int = 0, stream=None):
    """The log probability of each row's given token under the softmax of ``logits`` (rows, V), with
    the distribution's entropy and its ``top`` likeliest tokens.

    ``tokens`` (rows,) int32; one outside [0, V) stands for none: 0, without a gradient.  Returns
    (logprobs (rows,), lse (rows,), entropy (rows,), top_logprobs (rows, top), top_tokens (rows, top)
    int32), float32, the likeliest first, ties to the lower token; ``top`` is at most 32.  A NaN or +inf
    logit makes its row's results NaN, and NaN tokens lead its top.  The
    results carry no autograd history: ``token_logprobs_backward`` gives their gradient."""
    return (_binding or _load_binding()).token_logprobs(logits, tokens, top, stream)


def token_logprobs_backward(grad_logprobs, logits, tokens, lse, grad_entropy=None, entropy=None, stream=None):
    """The gradient of ``token_logprobs``' log probabilities, and of its entropies with
    ``grad_entropy`` (rows,) and the ``entropy`` it gave, with respect to its ``logits``: (rows, V) in
    the logits' dtype.  ``lse`` is the one it gave."""
    return (_binding or _load_binding()).token_logprobs_backward(grad_logprobs, logits, tokens, lse, grad_entropy, entropy,
                                                                 stream)


def expert_sort(experts, E: int, stream=None):
    """Ranks the choices ``experts`` (tokens, k) int32 of a gate of ``E`` experts (``route``'s) by
    expert, equal ones by token and choice; one outside [0, E) is no choice (a padded token).

    Returns (places (tokens, k) int32 -- each choice's rank, -1 for none -- and offsets (E + 1,)
    int32: each expert's first rank, then the number of choices)."""
    return (_binding or _load_binding()).expert_sort(experts, E, stream)


def expert_gather(x, places, offsets, quantise: bool = False, stream=None):
    """The rows of ``x`` (tokens, D) in the order of the experts: row ``places[t, i]`` of the result
    (tokens * k, D) is row t; rows behind the last choice are zeros.  Its gradient is
    ``expert_combine`` without weights.  With ``quantise`` the rows come in 8 bits, as
    ``quantise_blocks`` gives them: (codes, scales)."""
    return (_binding or _load_binding()).expert_gather(x, places, offsets, quantise, stream)


def expert_combine(y, places, weights=None, stream=None):
    """The experts' outputs ``y`` (tokens * k, D) back at their tokens: (tokens, D) sums of
    ``weights[t, i] * y[places[t, i]]`` (weights (tokens, k) float32, None: 1), in y's dtype.  Its
    gradient is ``expert_combine_backward``."""
    return (_binding or _load_binding()).expert_combine(y, places, weights, stream)


def expert_combine_backward(grad, y, places, offsets, weights, stream=None):
    """The gradients of ``expert_combine``'s result with respect to ``y`` and ``weights``, for its
    gradient ``grad`` (tokens, D): ((tokens * k, D) in y's dtype, zeros behind the last choice, and
    (tokens, k) float32)."""
    return (_binding or _load_binding()).expert_combine_backward(grad, y, places, offsets, weights, stream)


def quantise_blocks(x, block_rows: int = 1, stream=None):
    """``x`` (rows, K) or (matrices, rows, K) in 8 bits: (codes float8_e4m3fn of x's shape, scales
    float32), a scale for each ``block_rows`` (1 or 128) x 128 numbers, the least power of two that
    brings their largest to 448 or below.  A code stands for code * scale; infinities and NaN become NaN."""
    return (_binding or _load_binding()).quantise_blocks(x, block_rows, stream)


def expert_product(x, x_scales, w, w_scales, offsets=None, dtype=None, stream=None):
    """Rows sorted by expert times each expert's weights, both in 8 bits.

    ``x`` (rows, K) float8_e4m3fn and ``x_scales`` (rows, ceil(K / 128)) as ``expert_gather`` or
    ``quantise_blocks`` give them; ``w`` (experts, N, K) float8_e4m3fn with ``w_scales`` (experts,
    ceil(N / 128), ceil(K / 128)), any float32 scales; ``offsets`` (experts + 1,) int32, ``expert_sort``'s
    -- None, with w (N, K) or one expert, for all rows.  K is a multiple of 16.  Returns (rows, N) in
    ``dtype`` (bfloat16, the default, or float32); rows outside the offsets are zeros.  The weights
    are constants.  The gradient with respect to x is the same product: the outputs' gradient in 8 bits along N
    (``quantise_blocks(grad)``, N a multiple of 16), times w transposed -- codes and the 128 x 128 blocks' scales alike,
    ``w.transpose(1, 2).contiguous()`` and ``w_scales.transpose(1, 2).contiguous()``, laid out once."""
    ops = _binding or _load_binding()
    if dtype is not None and str(dtype) not in ("torch.bfloat16", "torch.float32"):
        raise TypeError(f"dtype: unsupported dtype {dtype}: bfloat16 and float32 only")
    return ops.cache_load(cache, scales, slots, str(dtype) == "torch.float32", stream)


def cache_attention(q, cache, scales, table, lens, indices=None, scale=None, stream=None):
    """Attention of each sequence's newest tokens ``q`` (B, Q, query heads, D) over a 4-bit cache.

    ``table`` (B, width) int32 holds the page of each run of ``page`` positions, ``lens`` (B,) int32
    the positions stored, the Q new ones among them: token i sees those below lens - (Q - 1 - i),
    or those of them that ``indices`` (B, Q, K) int32 lists (``topk``'s columns; -1 pads).  ``scale``
    is 1 / sqrt(D) by default.  Returns (out (B, Q, query heads, D) in q's dtype, lse (B, Q, query
    heads) float32); a token that sees nothing gives 0 and -inf."""
    return (_binding or _load_binding()).cache_attention(q, cache, scales, table, lens, indices, scale, stream)


# --------------------------------------------- behind the selections ----------------

def token_logprobs(logits, tokens, top: int = 0, stream=None):
    """The log probability of each row's given token under the softmax of ``logits`` (rows, V), with
    the distribution's entropy and its ``top`` likeliest tokens.

    ``tokens`` (rows,) int32; one outside [0, V) stands for none: 0, without a gradient.  Returns
    (logprobs (rows,), lse (rows,), entropy (rows,), top_logprobs (rows, top), top_tokens (rows, top)
    int32), float32, the likeliest first, ties to the lower token; ``top`` is at most 32.  A NaN or +inf
    logit makes its row's results NaN, and NaN tokens lead its top.  The
    results carry no autograd history: ``token_logprobs_backward`` gives their gradient."""
    return (_binding or _load_binding()).token_logprobs(logits, tokens, top, stream)


def token_logprobs_backward(grad_logprobs, logits, tokens, lse, grad_entropy=None, entropy=None, stream=None):
    """The gradient of ``token_logprobs``' log probabilities, and of its entropies with
    ``grad_entropy`` (rows,) and the ``entropy`` it gave, with respect to its ``logits``: (rows, V) in
    the logits' dtype.  ``lse`` is the one it gave."""
    return (_binding or _load_binding()).token_logprobs_backward(grad_logprobs, logits, tokens, lse, grad_entropy, entropy,
                                                                 stream)


def expert_sort(experts, E: int, stream=None):
    """Ranks the choices ``experts`` (tokens, k) int32 of a gate of ``E`` experts (``route``'s) by
    expert, equal ones by token and choice; one outside [0, E) is no choice (a padded token).

    Returns (places (tokens, k) int32 -- each choice's rank, -1 for none -- and offsets (E + 1,)
    int32: each expert's first rank, then the number of choices)."""
    return (_binding or _load_binding()).expert_sort(experts, E, stream)


def expert_gather(x, places, offsets, quantise: bool = False, stream=None):
    """The rows of ``x`` (tokens, D) in the order of the experts: row ``places[t, i]`` of the result
    (tokens * k, D) is row t; rows behind the last choice are zeros.  Its gradient is
    ``expert_combine`` without weights.  With ``quantise`` the rows come in 8 bits, as
    ``quantise_blocks`` gives them: (codes, scales)."""
    return (_binding or _load_binding()).expert_gather(x, places, offsets, quantise, stream)


def expert_combine(y, places, weights=None, stream=None):
    """The experts' outputs ``y`` (tokens * k, D) back at their tokens: (tokens, D) sums of
    ``weights[t, i] * y[places[t, i]]`` (weights (tokens, k) float32, None: 1), in y's dtype.  Its
    gradient is ``expert_combine_backward``."""
    return (_binding or _load_binding()).expert_combine(y, places, weights, stream)


def expert_combine_backward(grad, y, places, offsets, weights, stream=None):
    """The gradients of ``expert_combine``'s result with respect to ``y`` and ``weights``, for its
    gradient ``grad`` (tokens, D): ((tokens * k, D) in y's dtype, zeros behind the last choice, and
    (tokens, k) float32)."""
    return (_binding or _load_binding()).expert_combine_backward(grad, y, places, offsets, weights, stream)


def quantise_blocks(x, block_rows: int = 1, stream=None):
    """``x`` (rows, K) or (matrices, rows, K) in 8 bits: (codes float8_e4m3fn of x's shape, scales
    float32), a scale for each ``block_rows`` (1 or 128) x 128 numbers, the least power of two that
    brings their largest to 448 or below.  A code stands for code * scale; infinities and NaN become NaN."""
    return (_binding or _load_binding()).quantise_blocks(x, block_rows, stream)


def expert_product(x, x_scales, w, w_scales, offsets=None, dtype=None, stream=None):
    """Rows sorted by expert times each expert's weights, both in 8 bits.

    ``x`` (rows, K) float8_e4m3fn and ``x_scales`` (rows, ceil(K / 128)) as ``expert_gather`` or
    ``quantise_blocks`` give them; ``w`` (experts, N, K) float8_e4m3fn with ``w_scales`` (experts,
    ceil(N / 128), ceil(K / 128)), any float32 scales; ``offsets`` (experts + 1,) int32, ``expert_sort``'s
    -- None, with w (N, K) or one expert, for all rows.  K is a multiple of 16.  Returns (rows, N) in
    ``dtype`` (bfloat16, the default, or float32); rows outside the offsets are zeros.  The weights
    are constants: the gradient with respect to x is the same product of the outputs' gradient with
    w transposed, whose 128 x 128 blocks' scales are the transposed ones."""
    ops = _binding or _load_binding()
    if dtype is not None and str(dtype) not in ("torch.bfloat16", "torch.float32"):
        raise TypeError(f"dtype: unsupported dtype {dtype}: bfloat16 and float32 only")
    return ops.expert_product(x, x_scales, w, w_scales, offsets, str(dtype) == "torch.float32", stream)
