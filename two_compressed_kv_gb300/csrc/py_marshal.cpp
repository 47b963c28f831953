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
  decltype(&mkv_rope_multi) rope_multi;
  decltype(&mkv_norm_rope) norm_rope;
  decltype(&mkv_norm_rope_grad) norm_rope_grad;
  decltype(&mkv_norm_rope_grad_workspace) norm_rope_grad_workspace;
  decltype(&mkv_prefill) prefill;
  decltype(&mkv_prefill_workspace) prefill_workspace;
  decltype(&mkv_paged_attend) attend;
  decltype(&mkv_paged_attend_workspace) attend_workspace;
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

// Fills a call's workspace: a new tensor whose memory belongs to the launching
// stream and which *keep holds until the call is issued, or the caller's.
// False where the library refused the sizes.
template <typename Args>
bool workspace_of(const Launch& l, int dev, Args* a, uint64_t need, at::Tensor* keep) {
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

// The caller's workspace; false: there is none.
template <typename Args>
bool given_workspace(PyObject* o, int dev, Args* a) {
  if (o == Py_None) return false;
  const at::Tensor& t = tensor(o, "workspace");
  a->workspace = flat<void>(o, "workspace", dev, at::kByte, {t.numel()});
  a->workspace_bytes = (uint64_t)t.numel();
  return true;
}

template <typename Args, typename Size>
bool workspace(PyObject* o, const Launch& l, int dev, const mkv_paged_cache* c, Args* a, Size size, at::Tensor* keep) {
  if (given_workspace(o, dev, a)) return true;
  const uint64_t need = size(c, a);
  return need != 0 && workspace_of(l, dev, a, need, keep);
}
// For sizes of which 0 means that none is needed and UINT64_MAX that the library refused.
template <typename Args>
bool workspace_or_none(PyObject* o, const Launch& l, int dev, Args* a, uint64_t need, at::Tensor* keep) {
  if (given_workspace(o, dev, a)) return true;
  if (need == UINT64_MAX) return false;
  return need == 0 || workspace_of(l, dev, a, need, keep);
}

void strides3(const at::Tensor& t, int64_t* out) {
  for (int i = 0; i < 3; ++i) out[i] = t.stride(i);
}
int32_t size32(int64_t n, const char* name) {
  if (n > INT32_MAX) value_error(std::string(name) + " is too large");
  return (int32_t)n;
}
float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + " must be a number");
  }
  return (float)v;
}
void strides2(const at::Tensor& t, int64_t* out) {
  out[0] = t.stride(0);
  out[1] = t.stride(1);
}

// What rope and rope_multi have in common.
mkv_rope_args rope_args(const mkv_rope_plan* plan, PyObject* px, PyObject* pout, int* device) {
  const at::Tensor& x = tensor(px, "x");
  const at::Tensor& out = tensor(pout, "out");
  const int dev = *device = x.get_device();
  if (dev < 0) value_error("x must be on a CUDA device");
  if (x.dim() != 4 || x.size(3) != plan->head_dim)
    value_error("x must be [batch, tokens, heads, " + std::to_string(plan->head_dim) + "], got " + text(x.sizes()));
  mkv_rope_args a;
  std::memset(&a, 0, sizeof(a));
  a.dtype = dtype_of(x, "x");
  if (out.scalar_type() != x.scalar_type()) type_error("out must be " + name_of(x.scalar_type()) + ", got " + name_of(out.scalar_type()));
  a.x = rows(x, "x", dev, {x.size(0), x.size(1), x.size(2), x.size(3)});
  a.out = rows(out, "out", dev, {x.size(0), x.size(1), x.size(2), x.size(3)});
  strides3(x, a.x_stride);
  strides3(out, a.out_stride);
  if (x.size(0) > INT32_MAX || x.size(2) > INT32_MAX) value_error("x is too large");
  a.batch = (int32_t)x.size(0);
  a.tokens = x.size(1);
  a.heads = (int32_t)x.size(2);
  return a;
}

// rope(plan, x, pos, out, transposed, first_pos, stream) -> status
long rope(PyObject* const* v) {
  const mkv_rope_plan* plan = address<mkv_rope_plan>(v[0]);
  int dev = 0;
  mkv_rope_args a = rope_args(plan, v[1], v[3], &dev);
  if (v[2] != Py_None) {
    const at::Tensor& pos = tensor(v[2], "pos");
    if (pos.scalar_type() != at::kInt) type_error("pos must be Int, got " + name_of(pos.scalar_type()));
    a.pos = static_cast<const int32_t*>(rows(pos, "pos", dev, {a.batch, a.tokens}));
    a.pos_stride = pos.stride(0);
  }
  a.transposed = integer32(v[4], "transposed");
  a.first_pos = integer32(v[5], "first_pos");
  const Launch l(dev, v[6]);
  return lib.rope(plan, &a, l.stream);
}

// Positions [axes, batch, tokens] with a contiguous last dimension.
const int32_t* axes_pos(PyObject* o, int dev, int64_t axes, int64_t batch, int64_t tokens, int64_t* stride,
                        int64_t* axis_stride) {
  const at::Tensor& pos = tensor(o, "pos");
  if (pos.scalar_type() != at::kInt) type_error("pos must be Int, got " + name_of(pos.scalar_type()));
  void* p = rows(pos, "pos", dev, {axes, batch, tokens});
  *axis_stride = pos.stride(0);
  *stride = pos.stride(1);
  return static_cast<const int32_t*>(p);
}

// rope_multi(plan, axes, x, pos, out, transposed, stream) -> status
long rope_multi(PyObject* const* v) {
  const mkv_rope_plan* plan = address<mkv_rope_plan>(v[0]);
  const mkv_rope_axes* axes = address<mkv_rope_axes>(v[1]);
  int dev = 0;
  mkv_rope_args a = rope_args(plan, v[2], v[4], &dev);
  int64_t axis_stride = 0;
  a.pos = axes_pos(v[3], dev, axes->n_axes, a.batch, a.tokens, &a.pos_stride, &axis_stride);
  a.transposed = integer32(v[5], "transposed");
  const Launch l(dev, v[6]);
  return lib.rope_multi(plan, axes, &a, axis_stride, l.stream);
}

// norm_rope(plan, axes | None, pos, q, q_weight, q_out, k, k_weight, k_out, eps, weight_offset, first_pos, stream,
//           dq, dk, q_weight_grad, k_weight_grad, workspace) -> status; a gradient where dq is not None
long norm_rope(PyObject* const* v) {
  const mkv_rope_plan* plan = address<mkv_rope_plan>(v[0]);
  const mkv_rope_axes* axes = v[1] == Py_None ? nullptr : address<mkv_rope_axes>(v[1]);
  const bool grad = v[13] != Py_None;
  mkv_norm_rope_args a;
  std::memset(&a, 0, sizeof(a));
  const char* const names[2][5] = {{"q", "q_weight", "q_out", "dq", "q_weight_grad"}, {"k", "k_weight", "k_out", "dk", "k_weight_grad"}};
  int dev = -1;
  int wt = -1;
  at::ScalarType type = at::kFloat;
  for (int s = 0; s < 2; ++s) {
    PyObject* const* w = v + 3 + 3 * s;
    if (s == 1 && w[0] == Py_None) {
      if (w[1] != Py_None || w[2] != Py_None || v[14] != Py_None || v[16] != Py_None)
        value_error("k_weight, k_out, dk and k_weight_grad need k");
      break;
    }
    const at::Tensor& x = tensor(w[0], names[s][0]);
    if (s == 0) {
      dev = x.get_device();
      if (dev < 0) value_error("q must be on a CUDA device");
      type = x.scalar_type();
      a.dtype = dtype_of(x, "q");
      if (x.dim() != 4) value_error("q must be [batch, tokens, heads, head_dim]");
      a.batch = size32(x.size(0), "q");
      a.tokens = x.size(1);
    }
    if (x.dim() != 4) value_error("k must be [batch, tokens, heads, head_dim]");
    a.heads[s] = size32(x.size(2), names[s][0]);
    const std::initializer_list<int64_t> shape = {a.batch, a.tokens, a.heads[s], plan->head_dim};
    auto same = [&](const at::Tensor& t, const char* name) {
      if (t.scalar_type() != type) type_error(std::string(name) + " must be " + name_of(type) + ", got " + name_of(t.scalar_type()));
      return rows(t, name, dev, shape);
    };
    a.x[s] = same(x, names[s][0]);
    strides3(x, a.x_stride[s]);
    const at::Tensor& out = tensor(w[2], names[s][2]);
    a.out[s] = same(out, names[s][2]);
    strides3(out, a.out_stride[s]);
    if (w[1] != Py_None) {
      const at::Tensor& weight = tensor(w[1], names[s][1]);
      const int t = dtype_of(weight, names[s][1]);
      if (wt >= 0 && wt != t) type_error("q_weight and k_weight must be of one type");
      wt = t;
      a.weight[s] = rows(weight, names[s][1], dev, {plan->head_dim});
    }
    if (grad) {
      const at::Tensor& g = tensor(v[13 + s], names[s][3]);
      a.grad[s] = same(g, names[s][3]);
      strides3(g, a.grad_stride[s]);
      a.weight_grad[s] = flat<float>(v[15 + s], names[s][4], dev, at::kFloat, {plan->head_dim});
    }
  }
  a.weight_dtype = wt < 0 ? MKV_DT_F32 : wt;
  if (axes) {
    a.pos = axes_pos(v[2], dev, axes->n_axes, a.batch, a.tokens, &a.pos_stride, &a.pos_axis_stride);
  } else if (v[2] != Py_None) {
    const at::Tensor& pos = tensor(v[2], "pos");
    if (pos.scalar_type() != at::kInt) type_error("pos must be Int, got " + name_of(pos.scalar_type()));
    a.pos = static_cast<const int32_t*>(rows(pos, "pos", dev, {a.batch, a.tokens}));
    a.pos_stride = pos.stride(0);
  }
  a.eps = number(v[9], "eps");
  a.weight_offset = number(v[10], "weight_offset");
  a.first_pos = integer32(v[11], "first_pos");
  const Launch l(dev, v[12]);
  if (!grad) return lib.norm_rope(plan, axes, &a, l.stream);
  at::Tensor keep;
  const bool wants = a.weight_grad[0] || a.weight_grad[1];
  if (!given_workspace(v[17], dev, &a) && wants) {
    const uint64_t need = lib.norm_rope_grad_workspace(plan, &a);
    if (need == 0) return MKV_ERR_INVALID_ARG;
    workspace_of(l, dev, &a, need, &keep);
  }
  return lib.norm_rope_grad(plan, axes, &a, l.stream);
}

// prefill(q, k, v, out, lse, q_lens, kv_lens, prefix, docs, slopes, causal, window, scale, cap, workspace, stream,
//         status) -> status
long prefill(PyObject* const* v) {
  const at::Tensor &q = tensor(v[0], "q"), &k = tensor(v[1], "k"), &val = tensor(v[2], "v"), &out = tensor(v[3], "out");
  const int dev = q.get_device();
  if (dev < 0) value_error("q must be on a CUDA device");
  if (q.dim() != 4) value_error("q must be [batch, tokens, heads, head_dim]");
  if (k.dim() != 4) value_error("k must be [batch, kv_tokens, kv_heads, head_dim]");
  mkv_prefill_args a;
  std::memset(&a, 0, sizeof(a));
  a.dtype = dtype_of(q, "q", false);
  if (k.scalar_type() != q.scalar_type() || val.scalar_type() != q.scalar_type() || out.scalar_type() != q.scalar_type())
    type_error("q, k, v and out must be of one type");
  a.batch = size32(q.size(0), "q");
  a.q_tokens = q.size(1);
  a.n_q_heads = size32(q.size(2), "q");
  a.head_dim = size32(q.size(3), "q");
  a.kv_tokens = k.size(1);
  a.n_kv_heads = size32(k.size(2), "k");
  a.q = rows(q, "q", dev, {a.batch, a.q_tokens, a.n_q_heads, a.head_dim});
  a.k = rows(k, "k", dev, {a.batch, a.kv_tokens, a.n_kv_heads, a.head_dim});
  a.v = rows(val, "v", dev, {a.batch, a.kv_tokens, a.n_kv_heads, a.head_dim});
  a.out = rows(out, "out", dev, {a.batch, a.q_tokens, a.n_q_heads, a.head_dim});
  strides3(q, a.q_stride);
  strides3(k, a.k_stride);
  strides3(val, a.v_stride);
  strides3(out, a.out_stride);
  a.lse = flat<float>(v[4], "lse", dev, at::kFloat, {a.batch, a.q_tokens, a.n_q_heads});
  a.q_lens = flat<int32_t>(v[5], "q_lens", dev, at::kInt, {a.batch});
  a.kv_lens = flat<int32_t>(v[6], "kv_lens", dev, at::kInt, {a.batch});
  a.prefix = flat<int32_t>(v[7], "prefix", dev, at::kInt, {a.batch});
  if (v[8] != Py_None) {
    const at::Tensor& docs = tensor(v[8], "docs");
    if (docs.scalar_type() != at::kInt) type_error("docs must be Int, got " + name_of(docs.scalar_type()));
    a.docs = static_cast<const int32_t*>(rows(docs, "docs", dev, {a.batch, a.kv_tokens}));
    a.docs_stride = docs.stride(0);
  }
  a.slopes = flat<float>(v[9], "slopes", dev, at::kFloat, {a.n_q_heads});
  a.status = flat<int32_t>(v[16], "status", dev, at::kInt, {1});
  a.causal = integer32(v[10], "causal");
  a.window = integer32(v[11], "window");
  a.scale = number(v[12], "scale");
  a.cap = number(v[13], "cap");
  const Launch l(dev, v[15]);
  at::Tensor keep;
  if (!workspace_or_none(v[14], l, dev, &a, lib.prefill_workspace(&a), &keep)) return MKV_ERR_INVALID_ARG;
  return lib.prefill(&a, l.stream);
}

// attend(cache, dev, q, seq_lens, out, lse, new_lens, tree, slopes, max_len, window, scale, cap, workspace, stream)
//   -> status
long attend(PyObject* const* v) {
  const mkv_paged_cache* c = address<mkv_paged_cache>(v[0]);
  const int dev = integer32(v[1], "device");
  const at::Tensor &q = tensor(v[2], "q"), &out = tensor(v[4], "out");
  if (q.dim() != 4) value_error("q must be [batch, new_tokens, q_heads, head_dim]");
  mkv_paged_attend_args a;
  std::memset(&a, 0, sizeof(a));
  a.n = size32(q.size(1), "q");
  a.n_q_heads = size32(q.size(2), "q");
  a.q_dtype = dtype_of(q, "q", false);
  a.q = rows(q, "q", dev, {c->batch, a.n, a.n_q_heads, c->head_dim});
  strides3(q, a.q_stride);
  a.out = flat<void>(v[4], "out", dev, q.scalar_type(), {c->batch, a.n, a.n_q_heads, c->head_dim});
  tensor(v[3], "seq_lens");
  a.seq_lens = flat<int32_t>(v[3], "seq_lens", dev, at::kInt, {c->batch});
  a.lse = flat<float>(v[5], "lse", dev, at::kFloat, {c->batch, a.n, a.n_q_heads});
  a.new_lens = flat<int32_t>(v[6], "new_lens", dev, at::kInt, {c->batch});
  a.tree = reinterpret_cast<const uint64_t*>(flat<int64_t>(v[7], "tree", dev, at::kLong, {c->batch, a.n}));
  a.slopes = flat<float>(v[8], "slopes", dev, at::kFloat, {a.n_q_heads});
  a.max_len = integer(v[9]);
  a.window = integer32(v[10], "window");
  a.scale = number(v[11], "scale");
  a.cap = number(v[12], "cap");
  const Launch l(dev, v[14]);
  at::Tensor keep;
  if (!workspace_or_none(v[13], l, dev, &a, lib.attend_workspace(c, &a), &keep)) return MKV_ERR_INVALID_ARG;
  return lib.attend(c, &a, l.stream);
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
  a.scale = number(v[9], "scale");
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

// bind(addresses of the entry points)
long bind(PyObject* const* v) {
  lib.rope = reinterpret_cast<decltype(lib.rope)>(address<void>(v[0]));
  lib.append = reinterpret_cast<decltype(lib.append)>(address<void>(v[1]));
  lib.decode_workspace = reinterpret_cast<decltype(lib.decode_workspace)>(address<void>(v[2]));
  lib.decode = reinterpret_cast<decltype(lib.decode)>(address<void>(v[3]));
  lib.evict_workspace = reinterpret_cast<decltype(lib.evict_workspace)>(address<void>(v[4]));
  lib.evict = reinterpret_cast<decltype(lib.evict)>(address<void>(v[5]));
  lib.rope_multi = reinterpret_cast<decltype(lib.rope_multi)>(address<void>(v[6]));
  lib.norm_rope = reinterpret_cast<decltype(lib.norm_rope)>(address<void>(v[7]));
  lib.norm_rope_grad = reinterpret_cast<decltype(lib.norm_rope_grad)>(address<void>(v[8]));
  lib.norm_rope_grad_workspace = reinterpret_cast<decltype(lib.norm_rope_grad_workspace)>(address<void>(v[9]));
  lib.prefill = reinterpret_cast<decltype(lib.prefill)>(address<void>(v[10]));
  lib.prefill_workspace = reinterpret_cast<decltype(lib.prefill_workspace)>(address<void>(v[11]));
  lib.attend = reinterpret_cast<decltype(lib.attend)>(address<void>(v[12]));
  lib.attend_workspace = reinterpret_cast<decltype(lib.attend_workspace)>(address<void>(v[13]));
  return 0;
}

#define ENTRY(name, n) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(bind, 14), ENTRY(rope, 7), ENTRY(append, 13), ENTRY(decode, 12), ENTRY(evict, 17),
                         ENTRY(rope_multi, 7), ENTRY(norm_rope, 18), ENTRY(prefill, 17), ENTRY(attend, 15),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
