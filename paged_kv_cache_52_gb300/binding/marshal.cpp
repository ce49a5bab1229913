// Argument checks and marshalling of the speculative step's calls, as a CPython
// module (`paged_kv_cache_52_gb300._marshal`).
//
// A step of one user keeps the GPU busy for 1.5 us in most of these calls; the
// same checks made in the interpreter took 18 us on the GB300's host, the
// allocation of the result through the dispatcher 7 of them.  Here a check reads
// the tensor's own fields.  Each function checks the tensors' devices, types,
// shapes and strides (ValueError), allocates what it returns, and calls the C
// entry of pagedkv.h on the device's current stream.  It returns the results,
// or the entry's status when that is not PKV_OK.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "../../include/pagedkv.h"

namespace {

using at::Tensor;

struct Refused {
  std::string text;
};

[[noreturn]] void refuse(const char* name, const std::string& what) {
  throw Refused{std::string(name) + " must be " + what};
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, "a tensor");
  return THPVariable_Unpack(o);
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "bfloat16";
    case at::kFloat: return "float32";
    case at::kInt: return "int32";
    case at::kLong: return "int64";
    default: return "uint8";
  }
}

// The address of a contiguous tensor of this type and shape on GPU `dev`.
void* packed(PyObject* o, const char* name, at::ScalarType type, int dev,
             std::initializer_list<int64_t> shape) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev ||
      t.sizes() != at::IntArrayRef(shape) || !t.is_contiguous()) {
    std::string s;
    for (int64_t d : shape) s += (s.empty() ? "" : ", ") + std::to_string(d);
    refuse(name, std::string("a contiguous ") + type_name(type) + " tensor [" + s +
                     "] on one GPU with the others");
  }
  return t.data_ptr();
}

void* packed_or_null(PyObject* o, const char* name, at::ScalarType type, int dev,
                     std::initializer_list<int64_t> shape) {
  return o == Py_None ? nullptr : packed(o, name, type, dev, shape);
}

struct Pools {
  int dev;
  int layers;  // dim 0 of five-dimensional pools, else 1
  int64_t k_layer, v_layer;
  at::ScalarType type;
  pkv_cache_desc desc;
  void *k, *v;
};

Pools pools(PyObject* ko, PyObject* vo, bool allow_bf16, bool allow_fp8, bool allow_layers) {
  const Tensor& k = tensor(ko, "k_cache");
  const Tensor& v = tensor(vo, "v_cache");
  Pools p;
  if (!k.is_cuda() || !v.is_cuda() || v.get_device() != k.get_device())
    refuse("k_cache and v_cache", "CUDA tensors on one GPU");
  p.dev = k.get_device();
  p.type = k.scalar_type();
  if (v.scalar_type() != p.type || !((allow_bf16 && p.type == at::kBFloat16) ||
                                     (allow_fp8 && p.type == at::kByte)))
    refuse("k_cache and v_cache", allow_bf16 && allow_fp8 ? "bfloat16 or uint8 (e4m3 codes), alike"
                                  : allow_fp8             ? "uint8 (e4m3 codes)"
                                                          : "bfloat16");
  const int64_t dims = k.dim();
  if (v.sizes() != k.sizes() || !(dims == 4 || (allow_layers && dims == 5)))
    refuse("k_cache and v_cache", allow_layers ? "alike, [NB, 16, Hkv, d] or [layers, NB, 16, Hkv, d]"
                                               : "alike, [NB, 16, Hkv, d]");
  const int64_t first = dims - 4;
  int64_t stride = 1;
  for (int64_t i = dims - 1; i >= first; --i) {
    if (k.size(i) > INT32_MAX) refuse("pools", "of sizes below 2^31");
    // a dimension of one element has no stride to speak of
    if (k.size(i) != 1 && (k.stride(i) != stride || v.stride(i) != stride))
      refuse(allow_layers ? "each layer's pool" : "pools", "contiguous");
    stride *= k.size(i);
  }
  if (dims == 5 && (k.size(0) < 1 || k.size(0) > INT32_MAX)) refuse("pools", "of one layer or more");
  p.layers = dims == 5 ? int(k.size(0)) : 1;
  p.k_layer = dims == 5 ? k.stride(0) : 0;
  p.v_layer = dims == 5 ? v.stride(0) : 0;
  p.desc = pkv_cache_desc{int32_t(k.size(first)), int32_t(k.size(first + 1)),
                          int32_t(k.size(first + 2)), int32_t(k.size(first + 3))};
  p.k = k.data_ptr();
  p.v = v.data_ptr();
  return p;
}

// The token stride of x [T, heads, d] bf16 with contiguous rows.
int64_t token_rows(const Tensor& x, const char* name, int dev, int64_t T, int64_t heads,
                   int64_t d) {
  if (x.scalar_type() != at::kBFloat16 || !x.is_cuda() || x.get_device() != dev || x.dim() != 3 ||
      x.size(0) != T || x.size(1) != heads || x.size(2) != d)
    refuse(name, "a bfloat16 tensor [" + std::to_string(T) + ", " + std::to_string(heads) + ", " +
                     std::to_string(d) + "] on one GPU with the pools");
  if (T && (x.stride(2) != 1 || (heads > 1 && x.stride(1) != d)))
    refuse(name, "contiguous within each token's row");
  return T > 1 ? x.stride(0) : heads * d;  // the stride of a single token is not used
}

int count(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse(name, "below 2^31 rows");
  return int(n);
}

int64_t whole(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v > INT32_MAX || v < INT32_MIN) refuse(name, "a 32-bit integer");
  return v;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

// A result: the caller's tensor (checked), or a new one.
Tensor result(PyObject* o, const char* name, at::ScalarType type, int dev,
              std::initializer_list<int64_t> shape) {
  if (o == Py_None)
    return at::detail::empty_cuda(at::IntArrayRef(shape), type, at::Device(at::kCUDA, dev),
                                  std::nullopt);
  packed(o, name, type, dev, shape);
  return THPVariable_Unpack(o);
}

PyObject* give(PyObject* given, const Tensor& t) {
  if (given != Py_None) {
    Py_INCREF(given);
    return given;
  }
  return THPVariable_Wrap(t);
}

// Runs `call(stream)` on GPU dev's current stream, without the interpreter's
// lock: a full launch queue makes it wait.
template <typename F>
int launch(int dev, F&& call) {
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  int st;
  Py_BEGIN_ALLOW_THREADS st = call(stream);
  Py_END_ALLOW_THREADS return st;
}

// Every function: a fixed number of positional arguments, C++ exceptions and
// refusals turned into Python's.
template <Py_ssize_t N, PyObject* (*F)(PyObject* const*)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(a);
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

struct TreeBatch {
  int S;
  const int32_t *q_start, *lens;
};

TreeBatch tree_batch(PyObject* q_start, PyObject* lens, int dev) {
  const Tensor& l = tensor(lens, "context_lens");
  if (l.dim() != 1) refuse("context_lens", "[S]");
  const int64_t S = l.size(0);
  TreeBatch b;
  b.S = count(S, "context_lens");
  b.lens = static_cast<const int32_t*>(packed(lens, "context_lens", at::kInt, dev, {S}));
  b.q_start = static_cast<const int32_t*>(packed(q_start, "q_start", at::kInt, dev, {S + 1}));
  return b;
}

// [S, width] int32
const int32_t* table(PyObject* o, const char* name, int dev, int64_t S, int* width) {
  const Tensor& t = tensor(o, name);
  if (t.dim() != 2) refuse(name, "two-dimensional");
  *width = count(t.size(1), name);
  return static_cast<const int32_t*>(packed(o, name, at::kInt, dev, {S, t.size(1)}));
}

// q, k, v, positions, rope_table, slot_mapping, k_cache, v_cache, scales (None or
// a pair), q_weight, k_weight, eps, interleaved, out
PyObject* rope_append(PyObject* const* a) {
  const bool fp8 = a[8] != Py_None;
  const Pools p = pools(a[6], a[7], !fp8, fp8, false);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const Tensor& rope = tensor(a[4], "rope_table");
  if (q.dim() != 3) refuse("q", "[T, Hq, d]");
  if (rope.dim() != 2) refuse("rope_table", "[positions, rot]");
  const int64_t T = q.size(0), hq = q.size(1), hkv = p.desc.kv_heads, d = p.desc.d_head;
  const int64_t sq = token_rows(q, "q", p.dev, T, hq, d);
  const int64_t sk = token_rows(k, "k", p.dev, T, hkv, d);
  const int64_t sv = token_rows(v, "v", p.dev, T, hkv, d);
  const void* pos = packed(a[3], "positions", at::kLong, p.dev, {T});
  const void* slots = packed(a[5], "slot_mapping", at::kLong, p.dev, {T});
  const int64_t rows = rope.size(0), rot = rope.size(1);
  const void* tab = packed(a[4], "rope_table", at::kFloat, p.dev, {rows, rot});
  const void* qw = packed_or_null(a[9], "q_weight", at::kBFloat16, p.dev, {d});
  const void* kw = packed_or_null(a[10], "k_weight", at::kBFloat16, p.dev, {d});
  float k_scale = 1.f, v_scale = 1.f;
  if (fp8) {
    if (!PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 2) refuse("scales", "a pair");
    k_scale = float(real(PyTuple_GET_ITEM(a[8], 0)));
    v_scale = float(real(PyTuple_GET_ITEM(a[8], 1)));
  }
  const float eps = float(real(a[11]));
  const int inter = PyObject_IsTrue(a[12]);
  if (inter < 0) throw python_error();
  const int nq = count(hq, "q"), nrot = count(rot, "rope_table");
  const Tensor out = result(a[13], "out", at::kBFloat16, p.dev, {T, hq, d});
  const void *qp = q.data_ptr(), *kp = k.data_ptr(), *vp = v.data_ptr();
  void* op = out.data_ptr();
  const int st = launch(p.dev, [&](void* stream) {
    const auto* pp = static_cast<const int64_t*>(pos);
    const auto* sp = static_cast<const int64_t*>(slots);
    const auto* tp = static_cast<const float*>(tab);
    return fp8 ? pkv_qk_norm_rope_append_fp8(qp, sq, kp, sk, vp, sv, T, nq, pp, tp, rows, nrot,
                                             inter, qw, kw, eps, sp, op, p.k, p.v, p.desc, k_scale,
                                             v_scale, stream)
               : pkv_qk_norm_rope_append(qp, sq, kp, sk, vp, sv, T, nq, pp, tp, rows, nrot, inter,
                                         qw, kw, eps, sp, op, p.k, p.v, p.desc, stream);
  });
  return st == PKV_OK ? give(a[13], out) : PyLong_FromLong(st);
}

// parents, q_start, context_lens, max_q_len, tree_mask, positions
PyObject* tree_layout(PyObject* const* a) {
  const Tensor& parents = tensor(a[0], "parents");
  if (!parents.is_cuda() || parents.dim() != 1) refuse("parents", "a CUDA tensor [total]");
  const int dev = parents.get_device();
  const int64_t total = parents.size(0);
  const auto* pp = static_cast<const int32_t*>(packed(a[0], "parents", at::kInt, dev, {total}));
  const TreeBatch b = tree_batch(a[1], a[2], dev);
  const int most = int(whole(a[3], "max_q_len")), n = count(total, "parents");
  const Tensor mask = result(a[4], "tree_mask", at::kLong, dev, {total});
  const Tensor pos = result(a[5], "positions", at::kLong, dev, {total});
  const int st = launch(dev, [&](void* stream) {
    return pkv_draft_tree_layout(pp, b.q_start, b.S, n, most, b.lens,
                                 static_cast<uint64_t*>(mask.data_ptr()),
                                 static_cast<int64_t*>(pos.data_ptr()), stream);
  });
  if (st != PKV_OK) return PyLong_FromLong(st);
  PyObject* m = give(a[4], mask);
  PyObject* p = give(a[5], pos);
  PyObject* both = PyTuple_Pack(2, m, p);
  Py_XDECREF(m);
  Py_XDECREF(p);
  return both;
}

// q, q_start, tree_mask, k_cache, v_cache, block_tables, context_lens, scale, out,
// max_q_len, workspace, bf16 out
PyObject* tree_attention(PyObject* const* a) {
  const Pools p = pools(a[3], a[4], true, false, false);
  const Tensor& q = tensor(a[0], "q");
  if (q.dim() != 3) refuse("q", "[total, Hq, d]");
  const int64_t total = q.size(0), hq = q.size(1), d = p.desc.d_head;
  const void* qp = packed(a[0], "q", at::kBFloat16, p.dev, {total, hq, d});
  const TreeBatch b = tree_batch(a[1], a[6], p.dev);
  const auto* mask =
      static_cast<const uint64_t*>(packed(a[2], "tree_mask", at::kLong, p.dev, {total}));
  int width;
  const int32_t* tables = table(a[5], "block_tables", p.dev, b.S, &width);
  const float scale = float(real(a[7]));
  const int most = int(whole(a[9], "max_q_len"));
  const Tensor& ws = tensor(a[10], "workspace");
  const int64_t ws_bytes = ws.numel();
  void* wp = packed(a[10], "workspace", at::kByte, p.dev, {ws_bytes});
  const int bf16 = PyObject_IsTrue(a[11]);
  if (bf16 < 0) throw python_error();
  const int nt = count(total, "q"), nq = count(hq, "q");
  const Tensor out = result(a[8], "out", bf16 ? at::kBFloat16 : at::kFloat, p.dev, {total, hq, d});
  void* op = out.data_ptr();
  const int st = launch(p.dev, [&](void* stream) {
    return bf16 ? pkv_paged_tree_attention_bf16out(qp, b.q_start, b.S, nt, most, nq, mask, p.k,
                                                   p.v, p.desc, tables, width, b.lens, scale, op,
                                                   wp, size_t(ws_bytes), stream)
                : pkv_paged_tree_attention(qp, b.q_start, b.S, nt, most, nq, mask, p.k, p.v,
                                           p.desc, tables, width, b.lens, scale,
                                           static_cast<float*>(op), wp, size_t(ws_bytes), stream);
  });
  return st == PKV_OK ? give(a[8], out) : PyLong_FromLong(st);
}

// k_cache, v_cache, block_tables, context_lens, q_start, accepted, num_accepted,
// new_context_lens
PyObject* accept_rows(PyObject* const* a) {
  const Pools p = pools(a[0], a[1], true, true, true);
  const TreeBatch b = tree_batch(a[4], a[3], p.dev);
  int width, most;
  const int32_t* tables = table(a[2], "block_tables", p.dev, b.S, &width);
  const int32_t* path = table(a[5], "accepted", p.dev, b.S, &most);
  const auto* n = static_cast<const int32_t*>(packed(a[6], "num_accepted", at::kInt, p.dev, {b.S}));
  const Tensor lens = result(a[7], "new_context_lens", at::kInt, p.dev, {b.S});
  const int elem = p.type == at::kByte ? 1 : 2;
  auto* lp = static_cast<int32_t*>(lens.data_ptr());
  const int st = launch(p.dev, [&](void* stream) {
    return pkv_kv_accept_rows(p.k, p.k_layer, p.v, p.v_layer, p.layers, p.desc, elem, tables,
                              width, b.lens, b.q_start, b.S, path, most, n, lp, stream);
  });
  return st == PKV_OK ? give(a[7], lens) : PyLong_FromLong(st);
}

#define PKV_METHOD(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<n, name>)), \
   METH_FASTCALL, nullptr}

PyMethodDef methods[] = {PKV_METHOD(rope_append, 14), PKV_METHOD(tree_layout, 6),
                         PKV_METHOD(tree_attention, 12), PKV_METHOD(accept_rows, 8),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
