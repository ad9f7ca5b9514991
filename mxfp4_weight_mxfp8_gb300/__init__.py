"""GB300 (sm_103a) MXFP8-activation x MXFP4-weight top-16 MoE decode layer.

A thin ctypes binding over the C ABI declared in ``include/moe.h``: every
function here only marshals arguments (tensor or array -> pointer, torch
stream -> cudaStream_t) and raises ``MoeError`` on a non-zero status. All of
the layer's work runs in the library's CUDA kernels; there is no other path.
Importing fails loudly when the library has not been built
(``python -c "import __graft_entry__ as g; g.build()"``).
"""
from __future__ import annotations

import ctypes
import os

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
    "moe_route", "moe_kv_plan", "moe_kv_append", "moe_kv_attend", "moe_kv_sync_status", "KvCache", "SCORE_SOFTMAX", "SCORE_SIGMOID",
    "MOE_KV_WORKSPACE_BYTES", "MOE_KV_MAX_REQUESTS",
]

MOE_OK, MOE_ERR_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA = 0, 1, 2, 3
MOE_ERR_DEVICE_TIMEOUT, MOE_ERR_DEVICE_IDS, MOE_ERR_STATE = 4, 5, 6
MOE_NOALLOC_SCRATCH_BYTES = 8 << 20  # static scratch of moe_run_noalloc
TOPK, UNIT_ROWS, MAX_BATCH = 16, 8, 256
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
MOE_KV_WORKSPACE_BYTES = 32 << 20  # workspace of moe_kv_attend
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
def _want(call: str, ok: bool, what: str):
    if not ok:
        raise MoeError(MOE_ERR_ARG, call, what)


def _tensor(call: str, name: str, t, dtypes, shape=None, dense=True):
    """Check one device tensor (None in `shape`: any size) and give its address."""
    _want(call, t.is_cuda and t.dtype in dtypes, f"{name} must be a CUDA tensor of {dtypes}")
    if shape is not None:
        got = t.shape
        _want(call, len(got) == len(shape) and all(w is None or w == g for w, g in zip(shape, got)),
              f"{name} must have shape {shape}, not {tuple(got)}")
    _want(call, not dense or t.is_contiguous(), f"{name} must be contiguous")
    return t.data_ptr()


def _one_device(call: str, tensors, stream):
    """The stream to launch on: every tensor must lie on the current device."""
    import torch

    device = torch.cuda.current_device()
    for t in tensors:
        _want(call, t is None or t.device.index == device, f"every tensor must lie on the current device ({device})")
    return _stream(stream)


_TYPES: dict = {}


def _types():
    if not _TYPES:
        import torch

        _TYPES.update(logits={torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}, f32=(torch.float32,),
                      i32=(torch.int32,), i64=(torch.int64,), bf16=(torch.bfloat16,),
                      u8=(torch.uint8, torch.float8_e4m3fn), scale=(torch.uint8,))
    return _TYPES


def moe_route(logits, ids, weights, scoring: int = SCORE_SOFTMAX, bias=None, groups: int = 1, group_topk: int = 1,
              group_score: int = 1, renormalize: bool = True, scale: float = 1.0, stream=None):
    """Routing ids (int32 [T, k]) and weights (float32 [T, k]) of logits [T, E]; see include/moe.h."""
    call, ty = "moe_route", _types()
    kind = ty["logits"].get(logits.dtype)
    _want(call, kind is not None and logits.is_cuda, "logits must be a float32, bfloat16 or float16 CUDA tensor")
    _want(call, logits.dim() == 2 and ids.dim() == 2, "logits and ids must have two dimensions")
    tokens, experts = logits.shape
    topk = ids.shape[1]
    _want(call, logits.stride(1) == 1 or experts <= 1, "logits must have unit stride along the experts")
    r = _Route(logits.data_ptr(), max(logits.stride(0), experts) if tokens <= 1 else logits.stride(0),
               None if bias is None else _tensor(call, "bias", bias, ty["f32"], (experts,)),
               _tensor(call, "ids", ids, ty["i32"], (tokens, topk)),
               _tensor(call, "weights", weights, ty["f32"], (tokens, topk)), kind, tokens, experts, topk, scoring,
               groups, group_topk, group_score, int(bool(renormalize)), scale)
    return _check(_lib.moe_route(r, _one_device(call, (logits, ids, weights, bias), stream)), call)


def moe_kv_plan(context_lens, query_lens, page_tokens: int, block_table, free_pages, free_head, query_start, seq_lens,
                positions, slots, counts, stream=None):
    """Pages, lengths, positions and slots of a step's new tokens; see include/moe.h."""
    call, ty = "moe_kv_plan", _types()
    i32, requests, tokens = ty["i32"], context_lens.shape[0], positions.shape[0]
    _want(call, block_table.dim() == 2 and block_table.stride(1) == 1, "block_table must be rows of unit stride")
    width = block_table.shape[1]
    p = _KvPlan(_tensor(call, "context_lens", context_lens, i32, (requests,)),
                _tensor(call, "query_lens", query_lens, i32, (requests,)),
                _tensor(call, "free_pages", free_pages, i32, (None,)), _tensor(call, "free_head", free_head, i32, (1,)),
                _tensor(call, "block_table", block_table, i32, (requests, width), dense=False),
                max(block_table.stride(0), width) if requests <= 1 else block_table.stride(0),
                _tensor(call, "query_start", query_start, i32, (requests + 1,)),
                _tensor(call, "seq_lens", seq_lens, i32, (requests,)),
                _tensor(call, "positions", positions, i32, (tokens,)), _tensor(call, "slots", slots, ty["i64"], (tokens,)),
                _tensor(call, "counts", counts, i32, (4,)), requests, page_tokens, width, free_pages.shape[0], tokens)
    tensors = (context_lens, query_lens, free_pages, free_head, block_table, query_start, seq_lens, positions, slots,
               counts)
    return _check(_lib.moe_kv_plan(p, _one_device(call, tensors, stream)), call)


def _cache(call: str, cache):
    """The C description of a cache given as its tensors (k, v, k_scale, v_scale)."""
    ty = _types()
    k, v, ks, vs = cache
    _want(call, k.dim() == 4, "the cache's keys must be [pages, kv_heads, page_tokens, head_dim]")
    pages, heads, page, dim = k.shape
    return _KvCache(_tensor(call, "k cache", k, ty["u8"]), _tensor(call, "v cache", v, ty["u8"], tuple(k.shape)),
                    _tensor(call, "k_scale", ks, ty["scale"], (pages, heads)),
                    _tensor(call, "v_scale", vs, ty["scale"], (pages, heads)), pages, page, heads, dim)


def moe_kv_append(cache, k, v, slots, stream=None):
    """Quantize keys and values (bfloat16 [T, kv_heads, head_dim], any token and head strides) into a cache given as
    its tensors (k, v, k_scale, v_scale), at `slots`; see include/moe.h."""
    call, ty = "moe_kv_append", _types()
    c = _cache(call, cache)
    tokens = slots.shape[0]
    shape = (tokens, c.kv_heads, c.head_dim)
    kp, vp = (_tensor(call, n, x, ty["bf16"], shape, dense=False) for n, x in (("k", k), ("v", v)))
    _want(call, k.stride(2) == 1 and v.stride(2) == 1, "k and v must have unit stride along head_dim")
    return _check(_lib.moe_kv_append(c, kp, k.stride(0), k.stride(1), vp, v.stride(0), v.stride(1),
                                     _tensor(call, "slots", slots, ty["i64"], (tokens,)), tokens,
                                     _one_device(call, (*cache, k, v, slots), stream)), call)


def moe_kv_attend(cache, q, block_table, query_start, seq_lens, out, workspace, lse=None, scale=None, window: int = 0,
                  stream=None):
    """Causal attention of q (bfloat16 [T, q_heads, head_dim]) over the cache, into out and lse (float32 [T, q_heads]);
    scale None: head_dim ** -0.5. `workspace`: MOE_KV_WORKSPACE_BYTES of zeroed uint8; see include/moe.h."""
    call, ty = "moe_kv_attend", _types()
    i32, c = ty["i32"], _cache(call, cache)
    _want(call, q.dim() == 3, "q must be [tokens, q_heads, head_dim]")
    tokens, heads, dim = q.shape
    requests = seq_lens.shape[0]
    _want(call, block_table.dim() == 2 and block_table.stride(1) == 1, "block_table must be rows of unit stride")
    width = block_table.shape[1]
    b = _KvBatch(_tensor(call, "block_table", block_table, i32, (requests, width), dense=False),
                 max(block_table.stride(0), width) if requests <= 1 else block_table.stride(0),
                 _tensor(call, "query_start", query_start, i32, (requests + 1,)),
                 _tensor(call, "seq_lens", seq_lens, i32, (requests,)), width, requests, tokens)
    qp = _tensor(call, "q", q, ty["bf16"], (tokens, heads, c.head_dim), dense=False)
    _want(call, q.stride(2) == 1, "q must have unit stride along head_dim")
    _want(call, workspace.numel() * workspace.element_size() >= MOE_KV_WORKSPACE_BYTES,
          f"workspace must have {MOE_KV_WORKSPACE_BYTES} bytes")
    op = _tensor(call, "out", out, ty["bf16"], (tokens, heads, dim))
    lp = None if lse is None else _tensor(call, "lse", lse, ty["f32"], (tokens, heads))
    stream = _one_device(call, (*cache, q, block_table, query_start, seq_lens, out, workspace, lse), stream)
    return _check(_lib.moe_kv_attend(c, b, qp, q.stride(0), q.stride(1), heads, dim ** -0.5 if scale is None else scale,
                                     window, op, lp, workspace.data_ptr(), stream), call)


def moe_kv_sync_status(workspace, stream=None) -> int:
    """Device status of the finished moe_kv_attend calls on this workspace (not raised)."""
    return _lib.moe_kv_sync_status(_ptr(workspace), _stream(stream))


class KvCache:
    """A layer's paged cache: its tensors (e4m3 codes, E8M0 scales) and an attention workspace.

    ``append(k, v, slots)`` writes a step's keys and values, ``attend(q,
    block_table, query_start, seq_lens)`` returns the BF16 [T, q_heads,
    head_dim] outputs (and the FP32 log-sum-exp with ``return_lse=True``), both
    on the current torch stream. Layers that run one after the other on one
    stream can share a workspace.
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

        if out is None:
            out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device) if return_lse else None
        moe_kv_attend(self.tensors, q, block_table, query_start, seq_lens, out, self.workspace, lse, scale, window,
                      stream)
        return (out, lse) if return_lse else out


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
