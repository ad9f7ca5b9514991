"""GB300 (sm_103a) MXFP8-activation x MXFP4-weight top-16 MoE decode layer.

Next to the layer: routing (``moe_route``), norms (``moe_norm``), rotary positions
(``moe_rope``) and the paged 8-bit cache with its attention (``moe_kv_plan``,
``moe_kv_append``, ``moe_kv_attend``, ``KvCache``) and the pages that requests
share (``moe_kv_fork``, ``moe_kv_reclaim``, ``moe_kv_copy``).

A thin ctypes binding over the C ABI declared in ``include/moe.h``: every
function here only marshals arguments (tensor or array -> pointer, torch
stream -> cudaStream_t; the smallest operators by ``csrc/tensors.cpp``) and
raises ``MoeError`` on a non-zero status. All of
the layer's work runs in the library's CUDA kernels; there is no other path.
Importing fails loudly when the library has not been built
(``python -c "import __graft_entry__ as g; g.build()"``).
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import os
import struct

from .build import LIBRARY, TENSORS

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
    "moe_norm", "moe_norm_quantize", "moe_rope", "moe_rope_turns", "ROPE_LINEAR", "ROPE_BANDS", "ROPE_RAMP",
    "moe_kv_fork", "moe_kv_reclaim", "moe_kv_reclaim_bytes", "moe_kv_copy",
    "moe_kv_attend_shared", "moe_kv_shared_bytes", "MOE_KV_SHARED_HEADER",
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
MOE_KV_SHARED_HEADER = 65536  # moe_kv_attend_shared's scratch in front of the rows' outputs


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


class _Norm(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_stride", _i64), ("residual", _vp), ("residual_stride", _i64), ("residual_out", _vp),
                ("residual_out_stride", _i64), ("weight", _vp), ("out", _vp), ("out_stride", _i64), ("codes", _vp),
                ("scales", _vp)] + [(n, _i32) for n in ("dtype", "residual_dtype", "weight_dtype", "tokens", "hidden")] + [
                    ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float)]


class _Rope(ctypes.Structure):
    _fields_ = [("positions", _vp), ("turns", _vp)] + [
        (n + s, t) for n in ("q", "q_out", "k", "k_out")
        for s, t in (("", _vp), ("_token_stride", _i64), ("_head_stride", _i64))] + [
        (n, _i32) for n in ("tokens", "q_heads", "k_heads", "head_dim", "rotary_dim", "interleaved")] + [
        ("amplitude", ctypes.c_float)]


class _KvPrefixes(ctypes.Structure):
    _fields_ = [("group_start", _vp), ("prefix_lens", _vp), ("groups", _i32), ("least_tiles", _i32)]


class _KvFork(ctypes.Structure):
    _fields_ = [("parents", _vp), ("block_table", _vp), ("table_stride", _i64), ("seq_lens", _vp), ("free_pages", _vp),
                ("free_head", _vp), ("out_table", _vp), ("out_stride", _i64)] + [
        (n, _vp) for n in ("out_lens", "moves", "counts")] + [
        (n, _i32) for n in ("rows", "requests", "page_tokens", "table_width", "free_count")]


class _KvReclaim(ctypes.Structure):
    _fields_ = [("block_table", _vp), ("table_stride", _i64), ("seq_lens", _vp), ("free_pages", _vp), ("counts", _vp),
                ("out_table", _vp), ("out_stride", _i64), ("moves", _vp), ("workspace", _vp)] + [
        (n, _i32) for n in ("requests", "page_tokens", "table_width", "pages")]


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
        "moe_kv_shared_bytes": ([i32, i32, i32], ctypes.c_size_t),
        "moe_kv_attend_shared": ([ctypes.POINTER(_KvCache), ctypes.POINTER(_KvBatch), ctypes.POINTER(_KvPrefixes), vp, _i64, _i64,
                                  i32, ctypes.c_float, vp, vp, vp, vp, vp], i32),
        "moe_norm": ([ctypes.POINTER(_Norm), vp], i32),
        "moe_norm_quantize": ([vp, ctypes.POINTER(_Norm), vp], i32),
        "moe_rope": ([ctypes.POINTER(_Rope), vp], i32),
        "moe_rope_turns": ([i32, ctypes.c_double, i32] + [ctypes.c_double] * 4 + [vp], i32),
        "moe_kv_fork": ([ctypes.POINTER(_KvFork), vp], i32),
        "moe_kv_reclaim": ([ctypes.POINTER(_KvReclaim), vp], i32),
        "moe_kv_copy": ([ctypes.POINTER(_KvCache), vp, vp, i32, vp], i32),
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
_norm, _norm_quantize, _rope = (_packed(n) for n in ("moe_norm", "moe_norm_quantize", "moe_rope"))
_fork, _reclaim, _copy = (_packed(n) for n in ("moe_kv_fork", "moe_kv_reclaim", "moe_kv_copy"))
_attend_shared = _packed("moe_kv_attend_shared")
_torch = _native = None
_LOGITS: dict = {}


class _Declines:
    """In the place of csrc/tensors.cpp where that is not built, or not for this torch: it takes no call, so the checks here do."""

    def __getattr__(self, name):
        return lambda *_: None


def _use_torch():
    """torch and the lookups that need it, on the first call."""
    global _torch, _i32t, _i64t, _f32t, _bf16t, _u8t, _raw_stream, _native
    import torch

    native = _Declines()
    if TENSORS is not None and os.path.exists(TENSORS):
        loader = importlib.machinery.ExtensionFileLoader("_tensors", TENSORS)
        native = importlib.util.module_from_spec(importlib.util.spec_from_loader("_tensors", loader))
        loader.exec_module(native)
        native.bind(*(ctypes.cast(getattr(_lib, n), _vp).value for n in (
            "moe_norm", "moe_rope", "moe_kv_fork", "moe_kv_reclaim", "moe_kv_copy", "moe_kv_attend_shared")))
    _i32t, _i64t, _f32t, _bf16t, _u8t = torch.int32, torch.int64, torch.float32, torch.bfloat16, torch.uint8
    _LOGITS.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
    # The current stream's handle without building a stream object, where torch has it.
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    _torch, _native = torch, native
    return native


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


def _attend_args(call: str, cache, q, block_table, query_start, seq_lens, workspace, device: int):
    """(cache block, batch block, q's address and strides, tokens, heads, dim) of an attend call; the workspace checked."""
    block, _, dim = _cache_block(call, cache, device)
    requests = seq_lens.shape[0]
    table, table_stride, width = _table(call, block_table, requests, device)
    if q.dim() != 3:
        _refuse(call, "q must be [tokens, q_heads, head_dim]")
    tokens, heads, _ = q.shape
    batch = _BATCH.pack(table, table_stride, _dense(call, "query_start", query_start, _i32t, (requests + 1,), device),
                        _dense(call, "seq_lens", seq_lens, _i32t, (requests,), device), width, requests, tokens)
    room = workspace.shape
    if len(room) != 1 or room[0] < MOE_KV_WORKSPACE_BYTES:
        _refuse(call, f"workspace must be {MOE_KV_WORKSPACE_BYTES} bytes of uint8")
    return block, batch, _rows(call, "q", q, _bf16t, (tokens, heads, dim), device), tokens, heads, dim


def moe_kv_attend(cache, q, block_table, query_start, seq_lens, out, workspace, lse=None, scale=None, window: int = 0,
                  stream=None):
    """Causal attention of q (bfloat16 [T, q_heads, head_dim]) over the cache, into out and lse (float32 [T, q_heads]);
    scale None: head_dim ** -0.5. `workspace`: MOE_KV_WORKSPACE_BYTES of zeroed uint8; see include/moe.h."""
    call = "moe_kv_attend"
    device, stream = _on(call, q, stream)
    if not 0 <= window < 1 << 31:  # (ctypes would take it modulo 2^32)
        _refuse(call, "window must be 0 or a number of tokens below 2^31")
    block, batch, rows, tokens, heads, dim = _attend_args(call, cache, q, block_table, query_start, seq_lens, workspace, device)
    return _check(_attend(block, batch, *rows, heads, dim ** -0.5 if scale is None else scale, window,
                          _dense(call, "out", out, _bf16t, q.shape, device),
                          None if lse is None else _dense(call, "lse", lse, _f32t, (tokens, heads), device),
                          _dense(call, "workspace", workspace, _u8t, workspace.shape, device), stream), call)


def moe_kv_shared_bytes(tokens: int, q_heads: int, head_dim: int) -> int:
    """Bytes of moe_kv_attend_shared's scratch; 0 for arguments that the call refuses."""
    if not 0 <= min(tokens, q_heads, head_dim) <= max(tokens, q_heads, head_dim) < 1 << 31:  # (ctypes would take them modulo 2^32)
        return 0
    return _lib.moe_kv_shared_bytes(tokens, q_heads, head_dim)


def moe_kv_attend_shared(cache, q, block_table, query_start, seq_lens, group_start, prefix_lens, out, workspace, scratch,
                         lse=None, scale=None, least_tiles: int = 0, stream=None):
    """moe_kv_attend for requests in groups that share a prefix, whose pages are read once: group_start (int32 [G + 1]),
    prefix_lens (int32 [G]). `scratch`: uint8 of moe_kv_shared_bytes(T, q_heads, head_dim); see include/moe.h."""
    if stream is None:
        code = (_native or _use_torch()).attend_shared(cache, q, block_table, query_start, seq_lens, group_start, prefix_lens,
                                                       out, workspace, scratch, lse, scale, least_tiles)
        if code is not None:
            return _check(code, "moe_kv_attend_shared")
    call = "moe_kv_attend_shared"
    device, stream = _on(call, q, stream)
    block, batch, rows, tokens, heads, dim = _attend_args(call, cache, q, block_table, query_start, seq_lens, workspace, device)
    groups, room = prefix_lens.shape[0], scratch.shape
    if len(room) != 1 or room[0] < MOE_KV_SHARED_HEADER + 4 * tokens * heads * (dim + 1):
        _refuse(call, f"scratch must be {moe_kv_shared_bytes(tokens, heads, dim)} bytes of uint8")
    prefixes = _packed_args(call, _PREFIXES, _dense(call, "group_start", group_start, _i32t, (groups + 1,), device),
                            _dense(call, "prefix_lens", prefix_lens, _i32t, (groups,), device), groups, least_tiles)
    return _check(_attend_shared(block, batch, prefixes, *rows, heads, dim ** -0.5 if scale is None else scale,
                                 _dense(call, "out", out, _bf16t, q.shape, device),
                                 None if lse is None else _dense(call, "lse", lse, _f32t, (tokens, heads), device),
                                 _dense(call, "workspace", workspace, _u8t, workspace.shape, device),
                                 _dense(call, "scratch", scratch, _u8t, room, device), stream), call)


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


# --- norms, positions, shared pages ------------------------------------------
# On the current stream these go by _native (csrc/tensors.cpp), which answers None for arguments that it does not take;
# then, and on a given stream, by the checks here.
_NORM = struct.Struct("PqPqPqPPqPP5i2f0P")
_ROPE = struct.Struct("PP" + "PqqPqq" * 2 + "6if0P")
_FORK = struct.Struct("PPqPPPPqPPP5i0P")
_PREFIXES = struct.Struct("PP2i")
_RECLAIM = struct.Struct("PqPPPPqPP4i")


def _packed_args(call: str, block: struct.Struct, *values):
    """The C entry's argument block; refuses numbers that it has no room for."""
    try:
        return block.pack(*values)
    except (struct.error, OverflowError) as e:
        _refuse(call, f"a number out of range ({e})")


def _matrix(call: str, name: str, t, rows: int, columns: int, device: int):
    """(address, row stride) of a [rows, columns] tensor with unit stride along its rows."""
    if t.get_device() == device and t.dim() == 2:
        shape, (stride, unit) = t.shape, t.stride()
        if shape[0] == rows and shape[1] == columns and (unit == 1 or columns == 1):
            return t.data_ptr(), stride if rows > 1 else max(stride, columns)
    _refuse(call, f"{name} must be a tensor of shape ({rows}, {columns}) on cuda:{device} with unit stride along its rows, "
                  f"not {tuple(t.shape)} on {t.device}")


def _norm_block(call: str, x, weight, out, eps, residual, residual_out, codes, scales, weight_offset, device: int):
    if x.dim() != 2 or x.dtype not in _LOGITS or weight.dtype not in _LOGITS:
        _refuse(call, "x must be [tokens, hidden], x and weight float32, bfloat16 or float16")
    tokens, hidden = x.shape
    kind = 0
    for t in (residual, residual_out):
        if t is not None:
            kind = _LOGITS.get(t.dtype)
            if kind is None or (residual is not None and t.dtype is not residual.dtype):
                _refuse(call, "residual and residual_out must be of one type: float32, bfloat16 or float16")
    if out is not None and out.dtype is not x.dtype:
        _refuse(call, "out must be of x's type")
    none = (0, hidden)
    return _packed_args(
        call, _NORM, *_matrix(call, "x", x, tokens, hidden, device),
        *(none if residual is None else _matrix(call, "residual", residual, tokens, hidden, device)),
        *(none if residual_out is None else _matrix(call, "residual_out", residual_out, tokens, hidden, device)),
        _dense(call, "weight", weight, weight.dtype, (hidden,), device),
        *(none if out is None else _matrix(call, "out", out, tokens, hidden, device)),
        0 if codes is None else _dense(call, "codes", codes, _u8t, (tokens, hidden), device),
        0 if scales is None else _dense(call, "scales", scales, _u8t, (tokens, hidden // 32), device),
        _LOGITS[x.dtype], kind, _LOGITS[weight.dtype], tokens, hidden, eps, weight_offset)


def moe_norm(x, weight, out=None, eps: float = 1e-6, residual=None, residual_out=None, codes=None, scales=None,
             weight_offset: float = 0.0, stream=None):
    """Residual addition and root-mean-square norm of x [T, H] into out (x's type) and, in MXFP8, codes (uint8 [T, H])
    and scales (uint8 [T, H / 32]); x + residual into residual_out. See include/moe.h."""
    if stream is None:
        code = (_native or _use_torch()).norm(x, weight, out, eps, residual, residual_out, codes, scales, weight_offset)
        if code is not None:
            return _check(code, "moe_norm")
    call = "moe_norm"
    device, stream = _on(call, x, stream)
    return _check(_norm(_norm_block(call, x, weight, out, eps, residual, residual_out, codes, scales, weight_offset, device),
                        stream), call)


def moe_norm_quantize(handle, x, weight, out=None, eps: float = 1e-6, residual=None, residual_out=None,
                      weight_offset: float = 0.0, stream=None):
    """moe_norm whose MXFP8 output is the layer's activation plan (moe_group and moe_experts follow)."""
    call = "moe_norm_quantize"
    device, stream = _on(call, x, stream)
    return _check(_norm_quantize(handle, _norm_block(call, x, weight, out, eps, residual, residual_out, None, None,
                                                     weight_offset, device), stream), call)


ROPE_LINEAR, ROPE_BANDS, ROPE_RAMP = 0, 1, 2


def moe_rope_turns(rotary_dim: int, base: float = 10000.0, scaling: int = ROPE_LINEAR, factor: float = 1.0,
                   trained: float = 8192.0, low: float = 1.0, high: float = 4.0, device=None):
    """The table of moe_rope: int64 [rotary_dim / 2], angles of one position in units of 2^-64 turns; see include/moe.h."""
    import torch

    if not 0 <= min(rotary_dim, scaling) <= max(rotary_dim, scaling) < 1 << 31:  # (ctypes would take them modulo 2^32)
        _refuse("moe_rope_turns", "rotary_dim or scaling out of range")
    turns = torch.empty(max(rotary_dim // 2, 1), dtype=torch.int64)
    _check(_lib.moe_rope_turns(rotary_dim, base, scaling, factor, trained, low, high, turns.data_ptr()), "moe_rope_turns")
    return turns if device is None else turns.to(device)


def _heads(call: str, name: str, t, device: int):
    """(address, token stride, head stride, tokens, heads, dim) of a bfloat16 [tokens, heads, dim] tensor."""
    if t.dtype is _bf16t and t.get_device() == device and t.dim() == 3:
        (tokens, heads, dim), (token, head, unit) = t.shape, t.stride()
        if unit == 1:
            return t.data_ptr(), token if tokens > 1 else heads * dim, head if heads > 1 else dim, tokens, heads, dim
    _refuse(call, f"{name} must be a bfloat16 [tokens, heads, dim] tensor on cuda:{device} with unit stride along its last "
                  f"dimension, not {t.dtype} {tuple(t.shape)} on {t.device}")


def moe_rope(positions, turns, q, k=None, q_out=None, k_out=None, interleaved: bool = False, amplitude: float = 1.0, stream=None):
    """Rotates q and k (bfloat16 [T, heads, head_dim], any token and head strides) by `positions` into q_out and k_out,
    or in place; `turns`: moe_rope_turns on the device. See include/moe.h."""
    if stream is None:
        code = (_native or _use_torch()).rope(positions, turns, q, k, q_out, k_out, interleaved, amplitude)
        if code is not None:
            return _check(code, "moe_rope")
    call = "moe_rope"
    device, stream = _on(call, q, stream)
    *q_in, tokens, heads, dim = _heads(call, "q", q, device)
    q_to = q_in if q_out is None else _heads(call, "q_out", q_out, device)
    if q_out is not None and q_out.shape != q.shape:
        _refuse(call, "q_out must have q's shape")
    k_in = k_to = (0, 0, 0)
    k_heads = 0
    if k is not None:
        *k_in, k_tokens, k_heads, k_dim = _heads(call, "k", k, device)
        if k_tokens != tokens or k_dim != dim:
            _refuse(call, "k must have q's tokens and head_dim")
        k_to = k_in if k_out is None else _heads(call, "k_out", k_out, device)
        if k_out is not None and k_out.shape != k.shape:
            _refuse(call, "k_out must have k's shape")
    elif k_out is not None:
        _refuse(call, "k_out without k")
    pairs = turns.shape[0] if turns.dim() == 1 else 0
    block = _packed_args(call, _ROPE, _dense(call, "positions", positions, _i32t, (tokens,), device),
                         _dense(call, "turns", turns, _i64t, (pairs,), device), *q_in, *q_to[:3], *k_in, *k_to[:3], tokens, heads,
                         k_heads, dim, 2 * pairs, 1 if interleaved else 0, amplitude)
    return _check(_rope(block, stream), call)


def _moves(call: str, t, least: int, device: int):
    if t.dim() != 2 or t.shape[1] != 3 or t.shape[0] < least:
        _refuse(call, f"moves must be [{least} or more, 3]")
    return _dense(call, "moves", t, _i32t, t.shape, device)


def moe_kv_fork(parents, block_table, seq_lens, page_tokens: int, free_pages, free_head, out_table, out_lens, moves, counts,
                stream=None):
    """Rows of requests that go on from others' caches, and the moves that moe_kv_copy makes; see include/moe.h."""
    if stream is None:
        code = (_native or _use_torch()).fork(parents, block_table, seq_lens, page_tokens, free_pages, free_head, out_table, out_lens, moves, counts)
        if code is not None:
            return _check(code, "moe_kv_fork")
    call = "moe_kv_fork"
    device, stream = _on(call, parents, stream)
    requests, rows, free = parents.shape[0], seq_lens.shape[0], free_pages.shape[0]
    table, table_stride, width = _table(call, block_table, rows, device)
    out, out_stride, out_width = _table(call, out_table, requests, device)
    if out_width != width:
        _refuse(call, "out_table must be as wide as block_table")
    block = _packed_args(call, _FORK, _dense(call, "parents", parents, _i32t, (requests,), device), table, table_stride,
                         _dense(call, "seq_lens", seq_lens, _i32t, (rows,), device),
                         _dense(call, "free_pages", free_pages, _i32t, (free,), device),
                         _dense(call, "free_head", free_head, _i32t, (1,), device), out, out_stride,
                         _dense(call, "out_lens", out_lens, _i32t, (requests,), device),
                         _dense(call, "moves", moves, _i32t, (requests, 3), device),
                         _dense(call, "counts", counts, _i32t, (4,), device), rows, requests, page_tokens, width, free)
    return _check(_fork(block, stream), call)


def moe_kv_reclaim(block_table, seq_lens, page_tokens: int, free_pages, counts, workspace, out_table=None, moves=None,
                   stream=None):
    """The free list of a pool of free_pages.shape[0] pages; with out_table and moves, the pool compacted. `workspace`:
    uint8 of moe_kv_reclaim_bytes(pages). See include/moe.h."""
    if stream is None:
        code = (_native or _use_torch()).reclaim(block_table, seq_lens, page_tokens, free_pages, counts, workspace, out_table, moves)
        if code is not None:
            return _check(code, "moe_kv_reclaim")
    call = "moe_kv_reclaim"
    device, stream = _on(call, block_table, stream)
    requests, pages = seq_lens.shape[0], free_pages.shape[0]
    table, table_stride, width = _table(call, block_table, requests, device)
    out, out_stride, out_width = (0, 0, width) if out_table is None else _table(call, out_table, requests, device)
    if out_width != width:
        _refuse(call, "out_table must be as wide as block_table")
    room = workspace.shape
    if len(room) != 1 or room[0] < moe_kv_reclaim_bytes(pages):
        _refuse(call, f"workspace must be {moe_kv_reclaim_bytes(pages)} bytes of uint8")
    block = _packed_args(call, _RECLAIM, table, table_stride, _dense(call, "seq_lens", seq_lens, _i32t, (requests,), device),
                          _dense(call, "free_pages", free_pages, _i32t, (pages,), device),
                          _dense(call, "counts", counts, _i32t, (4,), device), out, out_stride,
                          0 if moves is None else _moves(call, moves, max(1, pages // 2), device),
                          _dense(call, "workspace", workspace, _u8t, room, device), requests, page_tokens, width, pages)
    return _check(_reclaim(block, stream), call)


def moe_kv_reclaim_bytes(pages: int) -> int:
    """Bytes of moe_kv_reclaim's workspace (MOE_KV_RECLAIM_BYTES)."""
    return 1024 + 8 * pages


def moe_kv_copy(cache, moves, count=None, stream=None):
    """Copies pages within a cache given as its uint8 tensors (k, v, k_scale, v_scale): moves (int32 [n, 3]: from, to,
    tokens), the first `count` (int32 [1]) of them or all; see include/moe.h."""
    if stream is None:
        code = (_native or _use_torch()).copy(cache, moves, count)
        if code is not None:
            return _check(code, "moe_kv_copy")
    call = "moe_kv_copy"
    device, stream = _on(call, moves, stream)
    return _check(_copy(_cache_block(call, cache, device)[0], _moves(call, moves, 0, device),
                        None if count is None else _dense(call, "count", count, _i32t, (1,), device), moves.shape[0], stream), call)


class KvCache:
    """A layer's paged cache: its tensors (e4m3 codes, E8M0 scales) and an attention workspace.

    ``append(k, v, slots)`` writes a step's keys and values, ``attend(q,
    block_table, query_start, seq_lens)`` returns the BF16 [T, q_heads,
    head_dim] outputs (and the FP32 log-sum-exp with ``return_lse=True``),
    ``attend_shared`` does it for groups of requests that share a prefix, and
    ``copy(moves)`` moves pages within it (moe_kv_fork, moe_kv_reclaim), all
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

    def attend_shared(self, q, block_table, query_start, seq_lens, group_start, prefix_lens, out=None, scale=None,
                      return_lse: bool = False, scratch=None, least_tiles: int = 0, stream=None):
        import torch

        if q.dim() != 3:
            _refuse("moe_kv_attend_shared", "q must be [tokens, q_heads, head_dim]")
        with _allocating_on(stream):
            if out is None:
                out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
            lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device) if return_lse else None
            if scratch is None:
                scratch = torch.empty(moe_kv_shared_bytes(*q.shape), dtype=torch.uint8, device=q.device)
        moe_kv_attend_shared(self.tensors, q, block_table, query_start, seq_lens, group_start, prefix_lens, out, self.workspace,
                             scratch, lse, scale, least_tiles, stream)
        return (out, lse) if return_lse else out

    def copy(self, moves, count=None, stream=None):
        moe_kv_copy(self.tensors, moves, count, stream)

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
