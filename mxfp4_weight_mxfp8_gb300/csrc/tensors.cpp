// The Python calls of the decode step's smaller operators, from torch tensors to
// the C entries without a Python step for each tensor: one look at a tensor from
// Python takes half a microsecond, and a call of a few microseconds has up to ten.
//
// Each function takes the arguments of the package's function of that name, fills
// the C entry's argument block and calls it on the device's current stream. It
// does so for tensors that are what the entry needs; for anything else it returns
// None and has done nothing, and the package's own checks say what is wrong. The C
// entries are bound by address (bind), so this module needs no library but torch.
#include <Python.h>

#include <algorithm>
#include <cmath>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe.h"

namespace {

struct Entries {
  decltype(&moe_norm) norm;
  decltype(&moe_rope) rope;
  decltype(&moe_kv_fork) fork;
  decltype(&moe_kv_reclaim) reclaim;
  decltype(&moe_kv_copy) copy;
  decltype(&moe_kv_attend_shared) attend_shared;
} g_entries{};

struct Unfit {};  // an argument that only the package's checks can judge

constexpr at::ScalarType kInt = at::kInt, kLong = at::kLong, kByte = at::kByte;

// One call's device, taken from its first tensor: the current one.
struct Device {
  int index = -1;

  const at::Tensor& tensor(PyObject* o) {
    if (!THPVariable_Check(o)) throw Unfit();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided || !t.is_cuda()) throw Unfit();
    if (index < 0) {
      index = t.get_device();
      if (index != static_cast<int>(c10::cuda::current_device())) throw Unfit();
    }
    if (t.get_device() != index) throw Unfit();
    return t;
  }
  // The address of a contiguous tensor of this type and shape.
  template <class T>
  T* dense(PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor& t = tensor(o);
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous()) throw Unfit();
    return static_cast<T*>(t.data_ptr());
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream(); }
};

int dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return MOE_F32;
    case at::kBFloat16: return MOE_BF16;
    case at::kHalf: return MOE_F16;
    default: throw Unfit();
  }
}

int narrow(int64_t n) {
  if (n < 0 || n > 0x7FFFFFFF) throw Unfit();
  return static_cast<int>(n);
}

int integer(PyObject* o) {
  const long v = PyLong_Check(o) ? PyLong_AsLong(o) : -1;
  if (v < 0 || v > 0x7FFFFFFF) {
    PyErr_Clear();
    throw Unfit();
  }
  return static_cast<int>(v);
}

float number(PyObject* o) {
  if (!PyFloat_Check(o)) throw Unfit();
  return static_cast<float>(PyFloat_AS_DOUBLE(o));
}

// A [rows, columns] tensor with unit stride along its rows.
struct Matrix {
  void* at = nullptr;
  int64_t stride = 0;
  int dtype = MOE_F32;
  Matrix(Device& d, PyObject* o, int64_t rows, int64_t columns) {
    stride = columns;
    if (o == Py_None) return;
    const at::Tensor& t = d.tensor(o);
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != columns || (t.stride(1) != 1 && columns != 1)) throw Unfit();
    at = t.data_ptr();
    dtype = dtype_of(t);
    stride = rows > 1 ? t.stride(0) : std::max(t.stride(0), columns);
  }
};

// A [tokens, heads, dim] BF16 tensor with unit stride along dim.
struct Heads {
  void* at = nullptr;
  int64_t token = 0, head = 0, tokens = 0, heads = 0, dim = 0;
  Heads(Device& d, PyObject* o) {
    if (o == Py_None) return;
    const at::Tensor& t = d.tensor(o);
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || t.stride(2) != 1) throw Unfit();
    at = t.data_ptr();
    tokens = t.size(0);
    heads = t.size(1);
    dim = t.size(2);
    token = tokens > 1 ? t.stride(0) : heads * dim;
    head = heads > 1 ? t.stride(1) : dim;
  }
  bool like(const Heads& o) const { return tokens == o.tokens && heads == o.heads && dim == o.dim; }
};

// An int32 block table of `rows` rows.
struct Table {
  int32_t* at;
  int64_t stride;
  int width;
  Table(Device& d, PyObject* o, int64_t rows) {
    const at::Tensor& t = d.tensor(o);
    if (t.scalar_type() != kInt || t.dim() != 2 || t.size(0) != rows || t.stride(1) != 1) throw Unfit();
    at = static_cast<int32_t*>(t.data_ptr());
    width = narrow(t.size(1));
    stride = rows > 1 ? t.stride(0) : std::max<int64_t>(t.stride(0), width);
  }
};

int64_t length(Device& d, PyObject* o) {
  const at::Tensor& t = d.tensor(o);
  if (t.dim() != 1) throw Unfit();
  return t.size(0);
}

moe_kv_cache_t cache_of(Device& d, PyObject* o) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) throw Unfit();
  const at::Tensor& k = d.tensor(PyTuple_GET_ITEM(o, 0));
  if (k.dim() != 4) throw Unfit();
  const int64_t scales[2] = {k.size(0), k.size(1)};
  moe_kv_cache_t c{};
  c.k = d.dense<uint8_t>(PyTuple_GET_ITEM(o, 0), kByte, k.sizes());
  c.v = d.dense<uint8_t>(PyTuple_GET_ITEM(o, 1), kByte, k.sizes());
  c.k_scale = d.dense<uint8_t>(PyTuple_GET_ITEM(o, 2), kByte, scales);
  c.v_scale = d.dense<uint8_t>(PyTuple_GET_ITEM(o, 3), kByte, scales);
  c.pages = narrow(k.size(0));
  c.kv_heads = narrow(k.size(1));
  c.page_tokens = narrow(k.size(2));
  c.head_dim = narrow(k.size(3));
  return c;
}

// Runs `body` on exactly kCount arguments: its status, or None where it does not fit.
template <int kCount, class F>
PyObject* call(PyObject* const* a, Py_ssize_t n, F&& body) {
  if (n == kCount) {
    try {
      Device d;
      return PyLong_FromLong(body(a, d));
    } catch (...) {  // Unfit, or torch's own, with or without a Python error
      PyErr_Clear();
    }
  }
  Py_RETURN_NONE;
}

// x, weight, out, eps, residual, residual_out, codes, scales, weight_offset
PyObject* norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call<9>(args, n, [](PyObject* const* a, Device& d) {
    const at::Tensor& x = d.tensor(a[0]);
    if (x.dim() != 2) throw Unfit();
    const int64_t tokens = x.size(0), hidden = x.size(1);
    const Matrix in(d, a[0], tokens, hidden), out(d, a[2], tokens, hidden), residual(d, a[4], tokens, hidden), to(d, a[5], tokens, hidden);
    const at::Tensor& w = d.tensor(a[1]);
    if (w.dim() != 1 || w.size(0) != hidden || !w.is_contiguous()) throw Unfit();
    if ((out.at && out.dtype != in.dtype) || (residual.at && to.at && residual.dtype != to.dtype)) throw Unfit();
    moe_norm_t b{};
    b.x = in.at;
    b.x_stride = in.stride;
    b.residual = residual.at;
    b.residual_stride = residual.stride;
    b.residual_out = to.at;
    b.residual_out_stride = to.stride;
    b.weight = w.data_ptr();
    b.out = out.at;
    b.out_stride = out.stride;
    const int64_t codes[2] = {tokens, hidden}, scales[2] = {tokens, hidden / 32};
    if (a[6] != Py_None) b.codes = d.dense<uint8_t>(a[6], kByte, codes);
    if (a[7] != Py_None) b.scales = d.dense<uint8_t>(a[7], kByte, scales);
    b.dtype = in.dtype;
    b.residual_dtype = residual.at ? residual.dtype : to.dtype;
    b.weight_dtype = dtype_of(w);
    b.tokens = narrow(tokens);
    b.hidden = narrow(hidden);
    b.eps = number(a[3]);
    b.weight_offset = number(a[8]);
    return g_entries.norm(&b, d.stream());
  });
}

// positions, turns, q, k, q_out, k_out, interleaved, amplitude
PyObject* rope(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call<8>(args, n, [](PyObject* const* a, Device& d) {
    const Heads q(d, a[2]), k(d, a[3]), q_to(d, a[4] == Py_None ? a[2] : a[4]), k_to(d, a[5] == Py_None ? a[3] : a[5]);
    if (!q.at || !q.like(q_to) || !k.like(k_to) || (k.at && (k.tokens != q.tokens || k.dim != q.dim))) throw Unfit();
    const int64_t pairs = length(d, a[1]);
    moe_rope_t b{};
    b.positions = d.dense<int32_t>(a[0], kInt, q.tokens);
    b.turns = reinterpret_cast<const uint64_t*>(d.dense<int64_t>(a[1], kLong, pairs));
    b.q = q.at;
    b.q_token_stride = q.token;
    b.q_head_stride = q.head;
    b.q_out = q_to.at;
    b.q_out_token_stride = q_to.token;
    b.q_out_head_stride = q_to.head;
    b.k = k.at;
    b.k_token_stride = k.token;
    b.k_head_stride = k.head;
    b.k_out = k_to.at;
    b.k_out_token_stride = k_to.token;
    b.k_out_head_stride = k_to.head;
    b.tokens = narrow(q.tokens);
    b.q_heads = narrow(q.heads);
    b.k_heads = narrow(k.heads);
    b.head_dim = narrow(q.dim);
    b.rotary_dim = narrow(2 * pairs);
    if (!PyBool_Check(a[6])) throw Unfit();
    b.interleaved = a[6] == Py_True;
    b.amplitude = number(a[7]);
    return g_entries.rope(&b, d.stream());
  });
}

// parents, block_table, seq_lens, page_tokens, free_pages, free_head, out_table, out_lens, moves, counts
PyObject* fork(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call<10>(args, n, [](PyObject* const* a, Device& d) {
    const int64_t requests = length(d, a[0]), rows = length(d, a[2]), free = length(d, a[4]), moves[2] = {requests, 3};
    const Table table(d, a[1], rows), out(d, a[6], requests);
    if (out.width != table.width) throw Unfit();
    moe_kv_fork_t b{};
    b.parents = d.dense<int32_t>(a[0], kInt, requests);
    b.block_table = table.at;
    b.table_stride = table.stride;
    b.seq_lens = d.dense<int32_t>(a[2], kInt, rows);
    b.free_pages = d.dense<int32_t>(a[4], kInt, free);
    b.free_head = d.dense<int32_t>(a[5], kInt, 1);
    b.out_table = out.at;
    b.out_stride = out.stride;
    b.out_lens = d.dense<int32_t>(a[7], kInt, requests);
    b.moves = d.dense<int32_t>(a[8], kInt, moves);
    b.counts = d.dense<int32_t>(a[9], kInt, 4);
    b.rows = narrow(rows);
    b.requests = narrow(requests);
    b.page_tokens = integer(a[3]);
    b.table_width = table.width;
    b.free_count = narrow(free);
    return g_entries.fork(&b, d.stream());
  });
}

// block_table, seq_lens, page_tokens, free_pages, counts, workspace, out_table, moves
PyObject* reclaim(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call<8>(args, n, [](PyObject* const* a, Device& d) {
    const int64_t requests = length(d, a[1]), pages = length(d, a[3]), room = length(d, a[5]);
    const Table table(d, a[0], requests);
    if (room < static_cast<int64_t>(MOE_KV_RECLAIM_BYTES(pages))) throw Unfit();
    moe_kv_reclaim_t b{};
    b.block_table = table.at;
    b.table_stride = table.stride;
    b.seq_lens = d.dense<int32_t>(a[1], kInt, requests);
    b.free_pages = d.dense<int32_t>(a[3], kInt, pages);
    b.counts = d.dense<int32_t>(a[4], kInt, 4);
    if (a[6] != Py_None) {
      const Table out(d, a[6], requests);
      if (out.width != table.width) throw Unfit();
      b.out_table = out.at;
      b.out_stride = out.stride;
    }
    if (a[7] != Py_None) {
      const at::Tensor& moves = d.tensor(a[7]);
      if (moves.dim() != 2 || moves.size(0) < std::max<int64_t>(1, pages / 2) || moves.size(1) != 3) throw Unfit();
      b.moves = d.dense<int32_t>(a[7], kInt, moves.sizes());
    }
    b.workspace = d.dense<uint8_t>(a[5], kByte, room);
    b.requests = narrow(requests);
    b.page_tokens = integer(a[2]);
    b.table_width = table.width;
    b.pages = narrow(pages);
    return g_entries.reclaim(&b, d.stream());
  });
}

// cache, moves, count
PyObject* copy(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call<3>(args, n, [](PyObject* const* a, Device& d) {
    const at::Tensor& moves = d.tensor(a[1]);
    if (moves.dim() != 2 || moves.size(1) != 3) throw Unfit();
    const moe_kv_cache_t cache = cache_of(d, a[0]);
    const int32_t* at = d.dense<int32_t>(a[1], kInt, moves.sizes());
    const int32_t* count = a[2] == Py_None ? nullptr : d.dense<int32_t>(a[2], kInt, 1);
    return g_entries.copy(&cache, at, count, narrow(moves.size(0)), d.stream());
  });
}

// cache, q, block_table, query_start, seq_lens, group_start, prefix_lens, out, workspace, scratch, lse, scale, least_tiles
PyObject* attend_shared(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call<13>(args, n, [](PyObject* const* a, Device& d) {
    const Heads q(d, a[1]);
    if (!q.at) throw Unfit();
    const moe_kv_cache_t cache = cache_of(d, a[0]);
    const int64_t requests = length(d, a[4]), groups = length(d, a[6]), room = length(d, a[8]), scratch = length(d, a[9]);
    const Table table(d, a[2], requests);
    if (q.dim != cache.head_dim || room < MOE_KV_WORKSPACE_BYTES || scratch < MOE_KV_SHARED_HEADER + 4 * q.tokens * q.heads * (q.dim + 1)) throw Unfit();
    moe_kv_batch_t b{};
    b.block_table = table.at;
    b.table_stride = table.stride;
    b.query_start = d.dense<int32_t>(a[3], kInt, requests + 1);
    b.seq_lens = d.dense<int32_t>(a[4], kInt, requests);
    b.table_width = table.width;
    b.requests = narrow(requests);
    b.tokens = narrow(q.tokens);
    moe_kv_prefixes_t p{};
    p.group_start = d.dense<int32_t>(a[5], kInt, groups + 1);
    p.prefix_lens = d.dense<int32_t>(a[6], kInt, groups);
    p.groups = narrow(groups);
    p.least_tiles = integer(a[12]);
    const int64_t rows[3] = {q.tokens, q.heads, q.dim}, sums[2] = {q.tokens, q.heads};
    void* out = d.dense<void>(a[7], at::kBFloat16, rows);
    float* lse = a[10] == Py_None ? nullptr : d.dense<float>(a[10], at::kFloat, sums);
    const float scale = a[11] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(q.dim))) : number(a[11]);
    return g_entries.attend_shared(&cache, &b, &p, q.at, q.token, q.head, narrow(q.heads), scale, out, lse,
                                   d.dense<void>(a[8], kByte, room), d.dense<void>(a[9], kByte, scratch), d.stream());
  });
}

// The C entries' addresses, in the order of Entries.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* at[6];
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes the addresses of six entries");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (at[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null entry");
      return nullptr;
    }
  }
  g_entries = {reinterpret_cast<decltype(&moe_norm)>(at[0]), reinterpret_cast<decltype(&moe_rope)>(at[1]),
               reinterpret_cast<decltype(&moe_kv_fork)>(at[2]), reinterpret_cast<decltype(&moe_kv_reclaim)>(at[3]),
               reinterpret_cast<decltype(&moe_kv_copy)>(at[4]), reinterpret_cast<decltype(&moe_kv_attend_shared)>(at[5])};
  Py_RETURN_NONE;
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {ENTRY(bind), ENTRY(norm), ENTRY(rope), ENTRY(fork), ENTRY(reclaim), ENTRY(copy), ENTRY(attend_shared), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&g_module); }
