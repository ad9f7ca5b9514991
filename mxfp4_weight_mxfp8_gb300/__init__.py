"""GB300 (sm_103a) MXFP8-activation x MXFP4-weight top-16 MoE decode layer.

Next to the layer: routing (``moe_route``) and the paged 8-bit cache with its
attention (``moe_kv_plan``, ``moe_kv_append``, ``moe_kv_attend``, ``KvCache``).

A thin ctypes binding over the C ABI declared in ``include/moe.h``: every
function here only marshals arguments (tensor or array -> pointer, torch
stream -> cudaStream_t) and raises ``MoeError`` on a non-zero status. All of
the layer's work runs in the library's CUDA kernels; there is no other path.
Importing fails loudly when the library has not been built
(``python -c "import __graft_entry__ as g; g.build()"``).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct

from .build import LIBRARY

__all__ = [
    "MoeError", "MoeInfo", "MoeLayer", "library", "moe_prepare", "moe_quantize", "moe_group",
    "moe_run", "moe_experts", "moe_run_noalloc", "moe_run_combined", "moe_run_host",
    "moe_sync_status", "moe_copy_plan", "moe_copy_units", "moe_copy_hidden", "moe_set_timeout",
    "moe_debug_withhold", "moe_debug_withhold_image", "moe_debug_paths", "moe_cluster_size", "moe_info",
    "moe_destroy", "moe_error_string",
    "MOE_OK", "MOE_ERR_ARG", "MOE_ERR_UNSUPPORTED", "MOE_ERR_CUDA", "MOE_ERR_DEVICE_TIMEOUT", "MOE_ERR_DEVICE_IDS",
    "MOE_ERR_STATE", "TOPK", "UNIT_ROWS", "MOE_NOALLOC_SCRATCH_BYTES", "moe_last_error_detail",
    "MAX_BATCH", "moe_device_supported", "moe_small_batch_build", "SMALL_NONE", "SMALL_PACKED", "SMALL_WIDE", "moe_debug_kernel_span", "moe_read_kernel_span",
    "moe_kernel_path", "PATH_GRID", "PATH_SMALL", "PATH_CLUSTER", "PATH_SMALL_WIDE",
    "moe_route", "moe_kv_plan", "moe_kv_append", "moe_kv_attend", "moe_kv_sync_status", "moe_kv_set_timeout", "moe_kv_debug_withhold", "KvCache", "SCORE_SOFTMAX", "SCORE_SIGMOID",
    "MOE_KV_WORKSPACE_BYTES", "MOE_KV_WORKSPACE_HEADER", "MOE_KV_MAX_REQUESTS",
]

MOE_OK, MOE_ERR_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA = 0, 1, 2, 3
MOE_ERR_DEVICE_TIMEOUT, MOE_ERR_DEVICE_IDS, MOE_ERR_STATE = 4, 5, 6
MOE_NOALLOC_SCRATCH_BYTES = 8 << 20  # static scratch of moe_run_noalloc
TOPK, UNIT_ROWS, MAX_BATCH = 16, 8, 256
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
MOE_KV_WORKSPACE_BYTES = 32 << 20  # workspace of moe_kv_attend
MOE_KV_WORKSPACE_HEADER = 8192  # its bytes that must start as zero
MOE_KV_MAX_REQUESTS = 1024


class MoeInfo(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_int), ("hidden", ctypes.c_int), ("inter", ctypes.c_int),
                ("hidden_floor_rule", ctypes.c_int), ("grid", ctypes.c_int),
                ("ring_stages", ctypes.c_int), ("smem_bytes", ctypes.c_int),
                ("stages_per_expert", ctypes.c_int), ("unit_capacity", ctypes.c_int),
                ("hidden_image_bytes", ctypes.c_int), ("weight_bytes", ctypes.c_size_t),
                ("workspace_bytes", ctypes.c_size_t)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64


class _Route(ctypes.Structure):
    _fields_ = [("logits", _vp), ("row_stride", _i64), ("bias", _vp), ("ids", _vp), ("weights", _vp)] + [
        (n, _i32) for n in ("dtype", "tokens", "experts", "topk", "scoring", "groups", "group_topk", "group_score",
                            "renormalize")] + [("scale", ctypes.c_float)]


class _KvPlan(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("context_lens", "query_lens", "free_pages", "free_head", "block_table")] + [
        ("table_stride", _i64)] + [(n, _vp) for n in ("query_start", "seq_lens", "positions", "slots", "counts")] + [
        (n, _i32) for n in ("requests", "page_tokens", "table_width", "free_count", "tokens")]


class _KvCache(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("k", "v", "k_scale", "v_scale")] + [
        (n, _i32) for n in ("pages", "page_tokens", "kv_heads", "head_dim")]


class _KvBatch(ctypes.Structure):
    _fields_ = [("block_table", _vp), ("table_stride", _i64), ("query_start", _vp), ("seq_lens", _vp)] + [
        (n, _i32) for n in ("table_width", "requests", "tokens")]


def _load():
    if not os.path.exists(LIBRARY):
        raise ImportError(f"CUDA library not built ({LIBRARY} missing): run "
                          "`python -c \"import __graft_entry__ as g; g.build()\"`")
    lib = ctypes.CDLL(LIBRARY)
    vp, i32, u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64
    signatures = {
        "moe_prepare": ([ctypes.POINTER(vp), vp, vp, vp, vp, i32, i32, i32], i32),
        "moe_quantize": ([vp, vp, i32, vp], i32),
        "moe_group": ([vp, vp, i32, vp], i32),
        "moe_run": ([vp, vp, vp, vp, i32, vp], i32),
        "moe_experts": ([vp, vp, i32, vp], i32),
        "moe_run_noalloc": ([vp, vp, vp, vp, i32, vp], i32),
        "moe_run_combined": ([vp, vp, vp, vp, vp, i32, vp], i32),
        "moe_run_host": ([vp, vp, vp, vp, i32, vp], i32),
        "moe_sync_status": ([vp, vp], i32),
        "moe_copy_plan": ([vp, vp, vp, i32], i32),
        "moe_copy_units": ([vp, vp, vp, vp, i32], i32),
        "moe_copy_hidden": ([vp, vp, vp, i32], i32),
        "moe_set_timeout": ([vp, u64], i32),
        "moe_debug_withhold": ([vp, i32], i32),
        "moe_debug_withhold_image": ([vp, i32], i32),
        "moe_debug_paths": ([vp, i32], i32),
        "moe_cluster_size": ([vp, i32], i32),
        "moe_kernel_path": ([vp, i32], i32),
        "moe_info": ([vp, ctypes.POINTER(MoeInfo)], i32),
        "moe_destroy": ([vp], None),
        "moe_error_string": ([i32], ctypes.c_char_p),
        "moe_last_error_detail": ([], ctypes.c_char_p),
        "moe_device_supported": ([i32, i32, ctypes.c_size_t], i32),
        "moe_small_batch_build": ([i32, i32, i32, i32, i32], i32),
        "moe_debug_kernel_span": ([vp, i32], i32),
        "moe_read_kernel_span": ([vp, ctypes.POINTER(u64)], i32),
        "moe_route": ([ctypes.POINTER(_Route), vp], i32),
        "moe_kv_plan": ([ctypes.POINTER(_KvPlan), vp], i32),
        "moe_kv_append": ([ctypes.POINTER(_KvCache), vp, _i64, _i64, vp, _i64, _i64, vp, i32, vp], i32),
        "moe_kv_sync_status": ([vp, vp], i32),
        "moe_kv_set_timeout": ([vp, u64, vp], i32),
        "moe_kv_debug_withhold": ([vp, i32, vp], i32),
        "moe_kv_attend": ([ctypes.POINTER(_KvCache), ctypes.POINTER(_KvBatch), vp, _i64, _i64, i32, ctypes.c_float,
                           i32, vp, vp, vp, vp], i32),
    }
    for name, (args, res) in signatures.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res
    return lib


_lib = _load()


def library():
    """The loaded ctypes library (its path is ``library()._name``)."""
    return _lib


class MoeError(RuntimeError):
    def __init__(self, code: int, call: str, detail: str | None = None):
        if detail is None:
            detail = _lib.moe_last_error_detail().decode()
        text = _lib.moe_error_string(code).decode()
        super().__init__(f"{call}: {text} (status {code}){': ' + detail if detail else ''}")
        self.code = code


def moe_last_error_detail() -> str:
    """Detail of this thread's last argument or CUDA error ("" if none)."""
    return _lib.moe_last_error_detail().decode()


def _check(code: int, call: str) -> int:
    if code != MOE_OK:
        raise MoeError(code, call)
    return code


def _ptr(obj):
    """Address of a torch tensor, numpy array or raw integer pointer."""
    if obj is None:
        return None
    if isinstance(obj, int):
        return obj
    if hasattr(obj, "data_ptr"):
        return obj.data_ptr()
    if hasattr(obj, "ctypes"):
        return obj.ctypes.data
    raise TypeError(f"cannot take the address of {type(obj).__name__}")


def _stream(stream):
    """cudaStream_t of a torch stream / raw handle; default: torch's current stream."""
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def moe_prepare(w13, s13, w2, s2, experts: int, hidden: int, inter: int):
    """Handle (an int) of a prepared layer; see include/moe.h."""
    handle = ctypes.c_void_p()
    _check(_lib.moe_prepare(ctypes.byref(handle), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2),
                            experts, hidden, inter), "moe_prepare")
    return handle.value


def moe_quantize(handle, x, batch: int, stream=None):
    return _check(_lib.moe_quantize(handle, _ptr(x), batch, _stream(stream)), "moe_quantize")


def moe_group(handle, ids, batch: int, stream=None):
    return _check(_lib.moe_group(handle, _ptr(ids), batch, _stream(stream)), "moe_group")


def moe_run(handle, x, ids, out, batch: int, stream=None):
    return _check(_lib.moe_run(handle, _ptr(x), _ptr(ids), _ptr(out), batch, _stream(stream)),
                  "moe_run")


def moe_experts(handle, out, batch: int, stream=None):
    return _check(_lib.moe_experts(handle, _ptr(out), batch, _stream(stream)), "moe_experts")


def moe_run_combined(handle, x, ids, weights, out, batch: int, stream=None):
    """moe_run, then out[t] = bf16(sum_s weights[t, s] * row[t, s]) (out: [B, H])."""
    return _check(_lib.moe_run_combined(handle, _ptr(x), _ptr(ids), _ptr(weights), _ptr(out),
                                        batch, _stream(stream)), "moe_run_combined")


def moe_run_noalloc(handle, x, ids, out, batch: int, stream=None):
    """moe_run with all per-call scratch in the library's static device
    buffer (for callers that cannot allocate when they run the layer)."""
    return _check(_lib.moe_run_noalloc(handle, _ptr(x), _ptr(ids), _ptr(out), batch,
                                       _stream(stream)), "moe_run_noalloc")


def moe_run_host(handle, x, ids, out, batch: int, stream=None):
    return _check(_lib.moe_run_host(handle, _ptr(x), _ptr(ids), _ptr(out), batch,
                                    _stream(stream)), "moe_run_host")


def moe_sync_status(handle, stream=None) -> int:
    """Device status of the finished calls (not raised: tests inspect it)."""
    return _lib.moe_sync_status(handle, _stream(stream))


def moe_copy_plan(handle, codes, scales, batch: int):
    return _check(_lib.moe_copy_plan(handle, _ptr(codes), _ptr(scales), batch), "moe_copy_plan")


def moe_copy_units(handle, count, experts, rows, capacity: int):
    return _check(_lib.moe_copy_units(handle, _ptr(count), _ptr(experts), _ptr(rows), capacity),
                  "moe_copy_units")


def moe_copy_hidden(handle, codes, scales, units: int):
    return _check(_lib.moe_copy_hidden(handle, _ptr(codes), _ptr(scales), units),
                  "moe_copy_hidden")


def moe_set_timeout(handle, nanoseconds: int):
    return _check(_lib.moe_set_timeout(handle, nanoseconds), "moe_set_timeout")


def moe_debug_withhold(handle, unit: int):
    return _check(_lib.moe_debug_withhold(handle, unit), "moe_debug_withhold")


def moe_debug_withhold_image(handle, unit: int):
    return _check(_lib.moe_debug_withhold_image(handle, unit), "moe_debug_withhold_image")


PATH_GRID, PATH_SMALL, PATH_CLUSTER, PATH_SMALL_WIDE = 0, 1, 2, 3


def moe_debug_paths(handle, path: int):
    """0 grid kernel, 1 small-batch kernel for 1-2 tokens (default), 2 cluster variant,
    3 small-batch kernel for up to 8 tokens."""
    return _check(_lib.moe_debug_paths(handle, path), "moe_debug_paths")


def moe_kernel_path(handle, batch: int) -> int:
    """The experts kernel a call of `batch` tokens runs on (PATH_*)."""
    n = _lib.moe_kernel_path(handle, batch)
    if n < 0:
        raise MoeError(-n, "moe_kernel_path")
    return n


def moe_debug_kernel_span(handle, enable: int):
    return _check(_lib.moe_debug_kernel_span(handle, enable), "moe_debug_kernel_span")


def moe_read_kernel_span(handle):
    """Span (ns) of the last experts-kernel launch recorded by the launch clock."""
    span = ctypes.c_uint64()
    _check(_lib.moe_read_kernel_span(handle, ctypes.byref(span)), "moe_read_kernel_span")
    return span.value


def moe_cluster_size(handle, batch: int) -> int:
    """CTAs per cluster a call of `batch` tokens runs on (0: the grid kernel)."""
    n = _lib.moe_cluster_size(handle, batch)
    if n < 0:
        raise MoeError(-n, "moe_cluster_size")
    return n


def moe_info(handle) -> MoeInfo:
    info = MoeInfo()
    _check(_lib.moe_info(handle, ctypes.byref(info)), "moe_info")
    return info


def moe_destroy(handle):
    _lib.moe_destroy(handle)


SMALL_NONE, SMALL_PACKED, SMALL_WIDE = 0, 1, 2


def moe_small_batch_build(experts: int, hidden: int, inter: int, batch: int, grid: int = 152) -> int:
    """The small-batch kernel's build for such a call (SMALL_*); no GPU needed."""
    n = _lib.moe_small_batch_build(experts, hidden, inter, batch, grid)
    if n < 0:
        raise MoeError(-n, "moe_small_batch_build")
    return n


def moe_device_supported(cc_major: int, cc_minor: int, smem_per_block_optin: int) -> int:
    """MOE_OK if a device with these properties runs the library (sm_103 with
    enough shared memory per block), else MOE_ERR_UNSUPPORTED."""
    return _lib.moe_device_supported(cc_major, cc_minor, smem_per_block_optin)


def moe_error_string(code: int) -> str:
    return _lib.moe_error_string(code).decode()


# --- the decode step around the layer ---------------------------------------
# These calls take torch tensors and are made for every layer of every step, so
# their host cost counts: each tensor is checked once, by the fewest calls, and
# the argument blocks are packed in one go (native alignment, as the C structs).
_ROUTE = struct.Struct("PqPPP9if")
_PLAN = struct.Struct("5Pq5P5i")
_CACHE = struct.Struct("4P4i")
_BATCH = struct.Struct("PqPP3i")


def _packed(name: str):
    """The C entry `name`, its argument blocks given as packed bytes."""
    fn, ref = _lib[name], getattr(_lib, name)
    fn.argtypes = [_vp if issubclass(t, ctypes._Pointer) else t for t in ref.argtypes]
    fn.restype = ref.restype
    return fn


_route, _plan, _append, _attend = (_packed(n) for n in ("moe_route", "moe_kv_plan", "moe_kv_append", "moe_kv_attend"))
_torch = None
_LOGITS: dict = {}


def _use_torch():
    """torch and the lookups that need it, on the first call."""
    global _torch, _i32t, _i64t, _f32t, _bf16t, _u8t, _raw_stream
    import torch

    _i32t, _i64t, _f32t, _bf16t, _u8t = torch.int32, torch.int64, torch.float32, torch.bfloat16, torch.uint8
    _LOGITS.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
    # The current stream's handle without building a stream object, where torch has it.
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    _torch = torch


def _refuse(call: str, what: str):
    raise MoeError(MOE_ERR_ARG, call, what)


def _dense(call: str, name: str, t, dtype, shape, device: int):
    """Address of a contiguous tensor of this type and shape on `device`."""
    if t.dtype is dtype and t.get_device() == device and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _refuse(call, f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{device}, "
                  f"not {t.dtype} {tuple(t.shape)} on {t.device}")


def _rows(call: str, name: str, t, dtype, shape, device: int):
    """(address, token stride, head stride) of a [tokens, heads, dim] tensor with unit stride along dim."""
    if t.dtype is dtype and t.get_device() == device and t.shape == shape:
        token, head, unit = t.stride()
        if unit == 1:
            return t.data_ptr(), token, head
    _refuse(call, f"{name} must be a {dtype} tensor of shape {tuple(shape)} on cuda:{device} with unit stride along its "
                  f"last dimension, not {t.dtype} {tuple(t.shape)} on {t.device}")


def _table(call: str, t, requests: int, device: int):
    """(address, row stride, width) of a block table."""
    if t.dtype is _i32t and t.get_device() == device and t.dim() == 2:
        rows, width = t.shape
        stride, unit = t.stride()
        if rows == requests and unit == 1:
            return t.data_ptr(), stride if requests > 1 else max(stride, width), width
    _refuse(call, f"block_table must be an int32 tensor of {requests} rows with unit stride on cuda:{device}")


def _on(call: str, t, stream) -> tuple:
    """(device, stream) of a call whose tensors lie where `t` does: the current device."""
    if _torch is None:
        _use_torch()
    device = t.get_device()
    if device < 0 or device != _torch.cuda.current_device():
        _refuse(call, f"tensors must lie on the current CUDA device, not on {t.device}")
    return device, _raw_stream(device) if stream is None else _stream(stream)


def moe_route(logits, ids, weights, scoring: int = SCORE_SOFTMAX, bias=None, groups: int = 1, group_topk: int = 1,
              group_score: int = 1, renormalize: bool = True, scale: float = 1.0, stream=None):
    """Routing ids (int32 [T, k]) and weights (float32 [T, k]) of logits [T, E]; see include/moe.h."""
    call = "moe_route"
    device, stream = _on(call, logits, stream)
    kind = _LOGITS.get(logits.dtype)
    if kind is None or logits.dim() != 2 or ids.dim() != 2:
        _refuse(call, "logits must be float32, bfloat16 or float16, logits and ids two-dimensional")
    tokens, experts = logits.shape
    row, unit = logits.stride()
    if unit != 1 and experts > 1:
        _refuse(call, "logits must have unit stride along the experts")
    shape = (tokens, ids.shape[1])
    block = _ROUTE.pack(
        logits.data_ptr(), row if tokens > 1 else max(row, experts),
        0 if bias is None else _dense(call, "bias", bias, _f32t, (experts,), device),
        _dense(call, "ids", ids, _i32t, shape, device), _dense(call, "weights", weights, _f32t, shape, device), kind,
        tokens, experts, shape[1], scoring, groups, group_topk, group_score, 1 if renormalize else 0, scale)
    return _check(_route(block, stream), call)


def moe_kv_plan(context_lens, query_lens, page_tokens: int, block_table, free_pages, free_head, query_start, seq_lens,
                positions, slots, counts, stream=None):
    """Pages, lengths, positions and slots of a step's new tokens; see include/moe.h."""
    call = "moe_kv_plan"
    device, stream = _on(call, context_lens, stream)
    requests, tokens, free = context_lens.shape[0], positions.shape[0], free_pages.shape[0]
    table, table_stride, width = _table(call, block_table, requests, device)
    per = (requests,)
    block = _PLAN.pack(
        _dense(call, "context_lens", context_lens, _i32t, per, device),
        _dense(call, "query_lens", query_lens, _i32t, per, device),
        _dense(call, "free_pages", free_pages, _i32t, (free,), device),
        _dense(call, "free_head", free_head, _i32t, (1,), device), table, table_stride,
        _dense(call, "query_start", query_start, _i32t, (requests + 1,), device),
        _dense(call, "seq_lens", seq_lens, _i32t, per, device),
        _dense(call, "positions", positions, _i32t, (tokens,), device),
        _dense(call, "slots", slots, _i64t, (tokens,), device),
        _dense(call, "counts", counts, _i32t, (4,), device), requests, page_tokens, width, free, tokens)
    return _check(_plan(block, stream), call)


def _cache_block(call: str, cache, device: int):
    """(packed description, kv_heads, head_dim) of a cache given as its tensors (k, v, k_scale, v_scale)."""
    k, v, k_scale, v_scale = cache
    shape = k.shape
    if len(shape) != 4:
        _refuse(call, "the cache's keys must be [pages, kv_heads, page_tokens, head_dim]")
    pages, heads, page, dim = shape
    scales = (pages, heads)
    return _CACHE.pack(_dense(call, "k cache", k, _u8t, shape, device), _dense(call, "v cache", v, _u8t, shape, device),
                       _dense(call, "k_scale", k_scale, _u8t, scales, device),
                       _dense(call, "v_scale", v_scale, _u8t, scales, device), pages, page, heads, dim), heads, dim


def moe_kv_append(cache, k, v, slots, stream=None):
    """Quantize keys and values (bfloat16 [T, kv_heads, head_dim], any token and head strides) into a cache given as
    its uint8 tensors (k, v, k_scale, v_scale), at `slots`; see include/moe.h."""
    call = "moe_kv_append"
    device, stream = _on(call, k, stream)
    block, heads, dim = _cache_block(call, cache, device)
    tokens = slots.shape[0]
    shape = (tokens, heads, dim)
    return _check(_append(block, *_rows(call, "k", k, _bf16t, shape, device), *_rows(call, "v", v, _bf16t, shape, device),
                          _dense(call, "slots", slots, _i64t, (tokens,), device), tokens, stream), call)


def moe_kv_attend(cache, q, block_table, query_start, seq_lens, out, workspace, lse=None, scale=None, window: int = 0,
                  stream=None):
    """Causal attention of q (bfloat16 [T, q_heads, head_dim]) over the cache, into out and lse (float32 [T, q_heads]);
    scale None: head_dim ** -0.5. `workspace`: MOE_KV_WORKSPACE_BYTES of zeroed uint8; see include/moe.h."""
    call = "moe_kv_attend"
    device, stream = _on(call, q, stream)
    block, _, dim = _cache_block(call, cache, device)
    requests = seq_lens.shape[0]
    table, table_stride, width = _table(call, block_table, requests, device)
    if q.dim() != 3:
        _refuse(call, "q must be [tokens, q_heads, head_dim]")
    tokens, heads, _ = q.shape
    shape = (tokens, heads, dim)
    batch = _BATCH.pack(table, table_stride, _dense(call, "query_start", query_start, _i32t, (requests + 1,), device),
                        _dense(call, "seq_lens", seq_lens, _i32t, (requests,), device), width, requests, tokens)
    if not 0 <= window < 1 << 31:  # (ctypes would take it modulo 2^32)
        _refuse(call, "window must be 0 or a number of tokens below 2^31")
    room = workspace.shape
    if len(room) != 1 or room[0] < MOE_KV_WORKSPACE_BYTES:
        _refuse(call, f"workspace must be {MOE_KV_WORKSPACE_BYTES} bytes of uint8")
    return _check(_attend(block, batch, *_rows(call, "q", q, _bf16t, shape, device), heads,
                          dim ** -0.5 if scale is None else scale, window, _dense(call, "out", out, _bf16t, shape, device),
                          None if lse is None else _dense(call, "lse", lse, _f32t, (tokens, heads), device),
                          _dense(call, "workspace", workspace, _u8t, room, device), stream), call)


def moe_kv_sync_status(workspace, stream=None) -> int:
    """Device status of the finished moe_kv_attend calls on this workspace (not raised)."""
    return _lib.moe_kv_sync_status(_ptr(workspace), _stream(stream))


def moe_kv_set_timeout(workspace, nanoseconds: int, stream=None):
    return _check(_lib.moe_kv_set_timeout(_ptr(workspace), nanoseconds, _stream(stream)), "moe_kv_set_timeout")


def moe_kv_debug_withhold(workspace, cta: int, stream=None):
    return _check(_lib.moe_kv_debug_withhold(_ptr(workspace), cta, _stream(stream)), "moe_kv_debug_withhold")


def _allocating_on(stream):
    """Context in which torch allocates for this stream (a torch stream or a raw handle); None: the current one."""
    if stream is None:
        return contextlib.nullcontext()
    if _torch is None:
        _use_torch()
    return _torch.cuda.stream(_torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


class KvCache:
    """A layer's paged cache: its tensors (e4m3 codes, E8M0 scales) and an attention workspace.

    ``append(k, v, slots)`` writes a step's keys and values, ``attend(q,
    block_table, query_start, seq_lens)`` returns the BF16 [T, q_heads,
    head_dim] outputs (and the FP32 log-sum-exp with ``return_lse=True``), both
    on the current torch stream or on ``stream``, which the outputs are then
    allocated for too (the inputs are the caller's to keep). Layers that run one after the other on one
    stream can share a workspace. ``status()`` synchronizes and returns the
    device status of the attend calls since it was last read: anything but
    MOE_OK and none of their outputs is to be used.
    """

    def __init__(self, pages: int, kv_heads: int, page_tokens: int = 64, head_dim: int = 128, device="cuda",
                 workspace=None):
        import torch

        codes = (pages, kv_heads, page_tokens, head_dim)
        self.k = torch.zeros(codes, dtype=torch.uint8, device=device)
        self.v = torch.zeros(codes, dtype=torch.uint8, device=device)
        self.k_scale = torch.zeros(codes[:2], dtype=torch.uint8, device=device)
        self.v_scale = torch.zeros(codes[:2], dtype=torch.uint8, device=device)
        if workspace is None:
            workspace = torch.zeros(MOE_KV_WORKSPACE_BYTES, dtype=torch.uint8, device=device)
        self.workspace = workspace

    @property
    def tensors(self):
        return self.k, self.v, self.k_scale, self.v_scale

    def append(self, k, v, slots, stream=None):
        moe_kv_append(self.tensors, k, v, slots, stream)

    def attend(self, q, block_table, query_start, seq_lens, out=None, scale=None, window: int = 0,
               return_lse: bool = False, stream=None):
        import torch

        with _allocating_on(stream):  # a block of the current stream's may still be in use there
            if out is None:
                out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
            lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device) if return_lse else None
        moe_kv_attend(self.tensors, q, block_table, query_start, seq_lens, out, self.workspace, lse, scale, window,
                      stream)
        return (out, lse) if return_lse else out

    def status(self, stream=None) -> int:
        return moe_kv_sync_status(self.workspace, stream)


class MoeLayer:
    """One prepared layer: owns a handle and allocates outputs with torch.

    ``weights`` = (w13, s13, w2, s2) uint8 tensors or arrays in the layout of
    include/moe.h (device or host). ``layer(x, ids)`` returns the BF16
    [B, 16, H] rows on x's device, on the current torch stream.
    """

    def __init__(self, weights):
        w13, s13, w2, s2 = weights
        experts, rows, half_hidden = (int(d) for d in w13.shape)
        self.experts, self.hidden, self.inter = experts, 2 * half_hidden, rows // 2
        self._keep = weights
        self.handle = moe_prepare(w13, s13, w2, s2, self.experts, self.hidden, self.inter)
        self._keep = None

    def __call__(self, x, ids, out=None, stream=None):
        import torch

        batch = int(x.shape[0])
        if out is None:
            out = torch.empty((batch, TOPK, self.hidden), dtype=torch.bfloat16, device=x.device)
        moe_run(self.handle, x, ids, out, batch, stream)
        return out

    def info(self) -> dict:
        return moe_info(self.handle).as_dict()

    def close(self):
        if self.handle:
            moe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
