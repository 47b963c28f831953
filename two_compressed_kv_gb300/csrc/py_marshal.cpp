// Argument marshalling of the rotary and paged-cache calls for Python: checks
// the tensors, fills the argument structs of include/mkv.h and calls the
// library.  A call from Python costs a few hundred nanoseconds here where the
// same checks cost 5 to 15 microseconds in Python, as much as the kernels of a
// small step take.  No arithmetic, no fallback, nothing kept between calls.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <initializer_list>
#include <string>

#include "mkv.h"

namespace {

// The library's entry points, set once by bind().
struct Entries {
  decltype(&mkv_rope) rope;
  decltype(&mkv_paged_append) append;
  decltype(&mkv_paged_decode_workspace) decode_workspace;
  decltype(&mkv_paged_decode) decode;
  decltype(&mkv_paged_evict_workspace) evict_workspace;
  decltype(&mkv_paged_evict) evict;
} lib;

struct Fail {
  PyObject* type;
  std::string text;
};
[[noreturn]] void type_error(const std::string& s) { throw Fail{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string& s) { throw Fail{PyExc_ValueError, s}; }

std::string name_of(at::ScalarType t) { return c10::toString(t); }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch tensor");
  return THPVariable_Unpack(o);
}

int dtype_of(const at::Tensor& t, const char* name, bool f32 = true) {
  switch (f32 || t.scalar_type() != at::kFloat ? t.scalar_type() : at::ScalarType::Undefined) {
    case at::kHalf: return MKV_DT_F16;
    case at::kBFloat16: return MKV_DT_BF16;
    case at::kFloat: return MKV_DT_F32;
    default: type_error(std::string(name) + " has type " + name_of(t.scalar_type()) + ", which the call does not take");
  }
}

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

// Address of a tensor of that shape on device `dev` whose last dimension is contiguous.
void* rows(const at::Tensor& t, const char* name, int dev, std::initializer_list<int64_t> shape) {
  if (t.get_device() != dev)
    value_error(std::string(name) + " is on " + t.device().str() + ", not on cuda:" + std::to_string(dev));
  const at::IntArrayRef want(shape.begin(), shape.size());
  if (t.sizes() != want) value_error(std::string(name) + " must have shape " + text(want) + ", got " + text(t.sizes()));
  if (!want.empty() && t.stride(-1) != 1 && want.back() > 1)
    value_error(std::string(name) + " must be contiguous in its last dimension");
  return t.data_ptr();
}

// Address of a contiguous tensor of that type and shape on device `dev`; None: NULL.
template <typename T>
T* flat(PyObject* o, const char* name, int dev, at::ScalarType type, std::initializer_list<int64_t> shape) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    type_error(std::string(name) + " must be " + name_of(type) + ", got " + name_of(t.scalar_type()));
  void* p = rows(t, name, dev, shape);
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return static_cast<T*>(p);
}

// As flat() for per-slot data [batch, kv_heads, slots]; *slots receives the row length.
template <typename T>
T* meta(PyObject* o, const char* name, int dev, at::ScalarType type, const mkv_paged_cache* c, int64_t* slots) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 3) value_error(std::string(name) + " must be [batch, kv_heads, slots]");
  *slots = t.size(2);
  return flat<T>(o, name, dev, type, {c->batch, c->n_kv_heads, t.size(2)});
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error("an integer argument is not a 64-bit integer");
  }
  return v;
}
int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " does not fit 32 bits");
  return (int32_t)v;
}
template <typename T>
T* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) {
    PyErr_Clear();
    type_error("an address is not an integer");
  }
  return static_cast<T*>(p);
}

// Device and stream of a call: the stream's address, or None for torch's current one.
struct Launch {
  c10::cuda::CUDAGuard guard;
  mkv_stream_t stream;
  bool given;
  Launch(int dev, PyObject* s) : guard((c10::DeviceIndex)dev), given(s != Py_None) {
    stream = given ? reinterpret_cast<mkv_stream_t>(address<void>(s))
                   : reinterpret_cast<mkv_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
  }
};

// Fills a call's workspace: the caller's tensor, or a new one whose memory
// belongs to the launching stream and which *keep holds until the call is issued.
// False where the library refused the sizes.
template <typename Args, typename Size>
bool workspace(PyObject* o, const Launch& l, int dev, const mkv_paged_cache* c, Args* a, Size size, at::Tensor* keep) {
  if (o != Py_None) {
    const at::Tensor& t = tensor(o, "workspace");
    a->workspace = flat<void>(o, "workspace", dev, at::kByte, {t.numel()});
    a->workspace_bytes = (uint64_t)t.numel();
    return true;
  }
  const uint64_t need = size(c, a);
  if (need == 0) return false;
  const auto options = at::TensorOptions().dtype(at::kByte).device(at::kCUDA, (c10::DeviceIndex)dev);
  if (l.given) {
    c10::cuda::CUDAStreamGuard on(
        c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(l.stream), (c10::DeviceIndex)dev));
    *keep = at::empty({(int64_t)need}, options);
  } else {
    *keep = at::empty({(int64_t)need}, options);
  }
  a->workspace = keep->data_ptr();
  a->workspace_bytes = need;
  return true;
}

void strides2(const at::Tensor& t, int64_t* out) {
  out[0] = t.stride(0);
  out[1] = t.stride(1);
}

// rope(plan, x, pos, out, transposed, first_pos, stream) -> status
long rope(PyObject* const* v) {
  const mkv_rope_plan* plan = address<mkv_rope_plan>(v[0]);
  const at::Tensor& x = tensor(v[1], "x");
  const at::Tensor& out = tensor(v[3], "out");
  const int dev = x.get_device();
  if (dev < 0) value_error("x must be on a CUDA device");
  if (x.dim() != 4 || x.size(3) != plan->head_dim)
    value_error("x must be [batch, tokens, heads, " + std::to_string(plan->head_dim) + "], got " + text(x.sizes()));
  mkv_rope_args a;
  std::memset(&a, 0, sizeof(a));
  a.dtype = dtype_of(x, "x");
  if (out.scalar_type() != x.scalar_type()) type_error("out must be " + name_of(x.scalar_type()) + ", got " + name_of(out.scalar_type()));
  a.x = rows(x, "x", dev, {x.size(0), x.size(1), x.size(2), x.size(3)});
  a.out = rows(out, "out", dev, {x.size(0), x.size(1), x.size(2), x.size(3)});
  for (int i = 0; i < 3; ++i) a.x_stride[i] = x.stride(i), a.out_stride[i] = out.stride(i);
  if (v[2] != Py_None) {
    const at::Tensor& pos = tensor(v[2], "pos");
    if (pos.scalar_type() != at::kInt) type_error("pos must be Int, got " + name_of(pos.scalar_type()));
    a.pos = static_cast<const int32_t*>(rows(pos, "pos", dev, {x.size(0), x.size(1)}));
    a.pos_stride = pos.stride(0);
  }
  if (x.size(0) > INT32_MAX || x.size(2) > INT32_MAX) value_error("x is too large");
  a.batch = (int32_t)x.size(0);
  a.tokens = x.size(1);
  a.heads = (int32_t)x.size(2);
  a.transposed = integer32(v[4], "transposed");
  a.first_pos = integer32(v[5], "first_pos");
  const Launch l(dev, v[6]);
  return lib.rope(plan, &a, l.stream);
}

// append(cache, dev, plan | None, k, v, slot, seq, pos, q, q_out, acc, pos_meta, stream) -> status
long append(PyObject* const* v) {
  const mkv_paged_cache* c = address<mkv_paged_cache>(v[0]);
  const int dev = integer32(v[1], "device");
  const mkv_rope_plan* plan = v[2] == Py_None ? nullptr : address<mkv_rope_plan>(v[2]);
  const at::Tensor &k = tensor(v[3], "k"), &val = tensor(v[4], "v");
  mkv_paged_append_args a;
  std::memset(&a, 0, sizeof(a));
  a.in_dtype = dtype_of(k, "k", false);
  if (k.dim() != 3) value_error("k must be [n, kv_heads, head_dim]");
  const int64_t n = a.n = k.size(0);
  if (val.scalar_type() != k.scalar_type()) type_error("k, v and q must be of one type");
  a.k = rows(k, "k", dev, {n, c->n_kv_heads, c->head_dim});
  a.v = rows(val, "v", dev, {n, c->n_kv_heads, c->head_dim});
  strides2(k, a.k_stride);
  strides2(val, a.v_stride);
  a.slot = flat<int32_t>(v[5], "slot", dev, at::kInt, {n});
  a.seq = flat<int32_t>(v[6], "seq", dev, at::kInt, {n});
  a.pos = flat<int32_t>(v[7], "pos", dev, at::kInt, {n});
  if (v[8] != Py_None) {
    const at::Tensor &q = tensor(v[8], "q"), &o = tensor(v[9], "q_out");
    if (q.scalar_type() != k.scalar_type()) type_error("k, v and q must be of one type");
    if (o.scalar_type() != q.scalar_type()) type_error("q_out must be " + name_of(q.scalar_type()) + ", got " + name_of(o.scalar_type()));
    if (q.dim() != 3) value_error("q must be [n, q_heads, head_dim]");
    const int64_t hq = q.size(1);
    if (hq > INT32_MAX) value_error("q has too many heads");
    a.q = rows(q, "q", dev, {n, hq, c->head_dim});
    a.q_out = rows(o, "q_out", dev, {n, hq, c->head_dim});
    a.n_q_heads = (int32_t)hq;
    strides2(q, a.q_stride);
    strides2(o, a.q_out_stride);
  } else if (v[9] != Py_None) {
    value_error("q_out needs q");
  }
  int64_t s0 = 0, s1 = 0;
  a.acc = meta<float>(v[10], "acc", dev, at::kFloat, c, &s0);
  a.pos_meta = meta<int32_t>(v[11], "pos_meta", dev, at::kInt, c, &s1);
  if (a.acc && a.pos_meta && s0 != s1) value_error("acc and pos_meta must have the same shape");
  a.meta_stride = a.acc ? s0 : s1;
  const Launch l(dev, v[12]);
  return lib.append(c, plan, &a, l.stream);
}

// decode(cache, dev, capacity, q, seq_lens, out, lse, acc, max_len, scale, workspace, stream) -> status
long decode(PyObject* const* v) {
  const mkv_paged_cache* c = address<mkv_paged_cache>(v[0]);
  const int dev = integer32(v[1], "device");
  const at::Tensor &q = tensor(v[3], "q"), &out = tensor(v[5], "out");
  if (q.dim() != 3) value_error("q must be [batch, q_heads, head_dim]");
  const int64_t hq = q.size(1);
  if (hq > INT32_MAX) value_error("q has too many heads");
  mkv_paged_decode_args a;
  std::memset(&a, 0, sizeof(a));
  a.n_q_heads = (int32_t)hq;
  a.q_dtype = dtype_of(q, "q", false);
  a.q = rows(q, "q", dev, {c->batch, hq, c->head_dim});
  strides2(q, a.q_stride);
  a.out_dtype = dtype_of(out, "out");
  a.out = flat<void>(v[5], "out", dev, out.scalar_type(), {c->batch, hq, c->head_dim});
  tensor(v[4], "seq_lens");
  a.seq_lens = flat<int32_t>(v[4], "seq_lens", dev, at::kInt, {c->batch});
  a.lse = flat<float>(v[6], "lse", dev, at::kFloat, {c->batch, hq});
  a.acc = meta<float>(v[7], "acc", dev, at::kFloat, c, &a.acc_stride);
  a.max_len = integer(v[8]);
  if (a.acc && a.max_len == 0) a.max_len = std::min(integer(v[2]), a.acc_stride);
  const double scale = PyFloat_AsDouble(v[9]);
  if (scale == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error("scale must be a number");
  }
  a.scale = (float)scale;
  const Launch l(dev, v[11]);
  at::Tensor keep;
  if (!workspace(v[10], l, dev, c, &a, lib.decode_workspace, &keep)) return MKV_ERR_INVALID_ARG;
  return lib.decode(c, &a, l.stream);
}

// evict(cache, dev, capacity, acc, pos, seq_lens, next_pos, budget, sink, recent, acc_out, pos_out, lens_out, src,
//       max_len, workspace, stream) -> status
long evict(PyObject* const* v) {
  const mkv_paged_cache* c = address<mkv_paged_cache>(v[0]);
  const int dev = integer32(v[1], "device");
  mkv_paged_evict_args a;
  std::memset(&a, 0, sizeof(a));
  tensor(v[3], "acc"), tensor(v[4], "pos"), tensor(v[5], "seq_lens"), tensor(v[6], "next_pos"), tensor(v[13], "src");
  a.acc = meta<float>(v[3], "acc", dev, at::kFloat, c, &a.meta_stride);
  a.pos = flat<int32_t>(v[4], "pos", dev, at::kInt, {c->batch, c->n_kv_heads, a.meta_stride});
  if ((v[10] == Py_None) != (v[11] == Py_None)) value_error("acc_out and pos_out go together");
  if (v[10] == Py_None) {
    a.acc_out = const_cast<float*>(a.acc);
    a.pos_out = const_cast<int32_t*>(a.pos);
    a.out_stride = a.meta_stride;
  } else {
    a.acc_out = meta<float>(v[10], "acc_out", dev, at::kFloat, c, &a.out_stride);
    a.pos_out = flat<int32_t>(v[11], "pos_out", dev, at::kInt, {c->batch, c->n_kv_heads, a.out_stride});
  }
  a.seq_lens = flat<int32_t>(v[5], "seq_lens", dev, at::kInt, {c->batch});
  a.next_pos = flat<int32_t>(v[6], "next_pos", dev, at::kInt, {c->batch});
  a.lens_out = v[12] == Py_None ? const_cast<int32_t*>(a.seq_lens)
                                : flat<int32_t>(v[12], "lens_out", dev, at::kInt, {c->batch});
  a.budget = integer32(v[7], "budget");
  a.sink = integer32(v[8], "sink");
  a.recent = integer32(v[9], "recent");
  a.src = flat<int32_t>(v[13], "src", dev, at::kInt, {c->batch, c->n_kv_heads, a.budget > 0 ? a.budget : 0});
  a.max_len = integer(v[14]);
  if (a.max_len == 0) a.max_len = std::min(integer(v[2]), a.meta_stride);
  const Launch l(dev, v[16]);
  at::Tensor keep;
  if (!workspace(v[15], l, dev, c, &a, lib.evict_workspace, &keep)) return MKV_ERR_INVALID_ARG;
  return lib.evict(c, &a, l.stream);
}

template <long (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(F(v));
  } catch (const Fail& f) {
    PyErr_SetString(f.type, f.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown failure in the marshalling of a call");
  }
  return nullptr;
}

// bind(addresses of the six entry points)
long bind(PyObject* const* v) {
  lib.rope = reinterpret_cast<decltype(lib.rope)>(address<void>(v[0]));
  lib.append = reinterpret_cast<decltype(lib.append)>(address<void>(v[1]));
  lib.decode_workspace = reinterpret_cast<decltype(lib.decode_workspace)>(address<void>(v[2]));
  lib.decode = reinterpret_cast<decltype(lib.decode)>(address<void>(v[3]));
  lib.evict_workspace = reinterpret_cast<decltype(lib.evict_workspace)>(address<void>(v[4]));
  lib.evict = reinterpret_cast<decltype(lib.evict)>(address<void>(v[5]));
  return 0;
}

#define ENTRY(name, n) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(bind, 6), ENTRY(rope, 7), ENTRY(append, 13), ENTRY(decode, 12), ENTRY(evict, 17),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
