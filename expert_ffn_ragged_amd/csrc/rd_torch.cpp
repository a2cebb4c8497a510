// Argument checks, output allocation and the current stream for the routed
// layer's entry points: a CPython module over librd.so and libtorch.
//
// Decode calls of these operators run 3 to 6 us on the GPU.  Checked in
// Python and called through ctypes they cost the host 9.3 us (route) to 11.2
// (group_rows), and the GPU waited; here it is 4.8 and 6.4.
// Every function takes its arguments by position (None for those not given)
// and the stream last; the Python functions of the same names hold the
// defaults and the documentation.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty_ops.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/StreamGuard.h>
#include <c10/core/impl/DeviceGuardImplInterface.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "rd.h"

namespace {

using at::Tensor;

PyObject* g_status_error = nullptr;  // the class of the exception for a nonzero status
PyObject* g_raw_stream = nullptr;    // device index -> the current stream's handle
PyObject* g_out_of_memory = nullptr; // torch's exception for a failed allocation

struct Refusal {
  PyObject* type;
  std::string what;
};
struct Status {
  int code;
};
struct PythonError {};  // already set

[[noreturn]] void wrong_type(const std::string& what) { throw Refusal{PyExc_TypeError, what}; }
[[noreturn]] void wrong_value(const std::string& what) { throw Refusal{PyExc_ValueError, what}; }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) wrong_type(std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

std::string type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return at::toString(t);
  }
}

const Tensor& need(PyObject* o, const char* name, at::ScalarType type, int ndim = -1) {
  const Tensor& t = tensor(o, name);
  if (!t.is_cuda()) wrong_value(std::string(name) + " must be on the GPU");
  if (t.scalar_type() != type)
    wrong_type(std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
  if (ndim >= 0 && t.dim() != ndim) wrong_value(std::string(name) + " must have " + std::to_string(ndim) + " dims");
  if (!t.is_contiguous()) wrong_value(std::string(name) + " must be contiguous");
  return t;
}

const Tensor& given(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
  const Tensor& t = need(o, name, type, static_cast<int>(shape.size()));
  if (t.sizes() != shape) {
    std::string want = std::string(name) + " must be [", got = "], got [";
    for (size_t i = 0; i < shape.size(); ++i) {
      want += (i ? ", " : "") + std::to_string(shape[i]);
      got += (i ? ", " : "") + std::to_string(t.size(i));
    }
    wrong_value(want + got + "]");
  }
  return t;
}

// bf16 or float32
at::ScalarType float_type(PyObject* o, const char* name) {
  const at::ScalarType t = tensor(o, name).scalar_type();
  if (t != at::kBFloat16 && t != at::kFloat)
    wrong_type(std::string(name) + " must be bfloat16 or float32, got " + type_name(t));
  return t;
}
int32_t rd_type(at::ScalarType t) { return t == at::kFloat ? RD_F32 : RD_BF16; }

// 4 for packed E2M1 codes, 8 for E4M3 ones
int code_bits(PyObject* o, const char* name) {
  const at::ScalarType t = tensor(o, name).scalar_type();
  if (t == at::kByte) return 4;
  if (t == at::kFloat8_e4m3fn) return 8;
  wrong_type(std::string(name) + " must be uint8 (two 4-bit codes a byte) or float8_e4m3fn, got " + type_name(t));
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}
int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v != static_cast<int32_t>(v)) wrong_value(std::string(name) + " must fit 32 bits");
  return static_cast<int32_t>(v);
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return static_cast<float>(v);
}
bool none(PyObject* o) { return o == Py_None; }

// Counts that size an output are checked before it is allocated, with the library's own statuses.
void in_range(int64_t v, int64_t most, int64_t supported) {
  if (v < 1 || v > most) throw Status{RD_EINVAL};
  if (v > supported) throw Status{RD_EUNSUPPORTED};
}

// One call: the GPU that its tensors live on, its stream, and the outputs it makes.
class Call {
 public:
  explicit Call(PyObject* stream) : stream_(stream) {}

  // Registers a tensor of the call and gives its address.
  void* at(const Tensor& t) {
    const int d = t.get_device();
    if (dev_ < 0) dev_ = d;
    if (d != dev_)
      wrong_value("operands on cuda:" + std::to_string(dev_) + " and cuda:" + std::to_string(d) +
                  ": every tensor of a call must be on one GPU");
    return t.data_ptr();
  }
  const int32_t* scalar(PyObject* o, const char* name) {  // a device scalar, or null for None
    if (none(o)) return nullptr;
    const Tensor& t = need(o, name, at::kInt);
    if (t.numel() != 1) wrong_value(std::string(name) + " must hold exactly one int32");
    return static_cast<const int32_t*>(at(t));
  }
  // The caller's tensor of this type and shape, or a new one beside ``like``.
  Tensor out(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, const Tensor& like) {
    if (!none(o)) return given(o, name, type, shape);
    if (none(stream_)) return make(type, shape, like);
    // From the given stream's memory: that of the current stream may still be in use by work that was queued there
    // before its tensor was freed, and nothing orders this call after that work.  The caller goes on with the tensor
    // on the current stream, so the allocator waits for that one too when it is freed.
    const c10::Stream s = given_stream();
    if (s.device_index() != like.get_device()) wrong_stream(s.device_index(), like.get_device());
    const c10::Stream current = c10::impl::getDeviceGuardImpl(c10::DeviceType::CUDA)->getStream(like.device());
    Tensor t;
    {
      c10::StreamGuard guard(s);
      t = make(type, shape, like);
    }
    if (current != s) t.record_stream(current);
    return t;
  }
  // Calls fn(stream), with the tensors' GPU made current (the library sizes its grids on the current device).
  template <class F>
  void launch(const F& fn) {
    void* handle;
    if (none(stream_)) {
      PyObject* index = PyLong_FromLong(dev_);
      handle = pointer(index == nullptr ? nullptr : PyObject_CallOneArg(g_raw_stream, index));
      Py_XDECREF(index);
    } else {
      const long d = attribute("device_index");
      if (d != dev_) wrong_stream(d, dev_);
      handle = pointer(PyObject_GetAttrString(stream_, "cuda_stream"));
    }
    check(handle, fn);
  }

 private:
  static void* pointer(PyObject* o) {
    if (o == nullptr) throw PythonError{};
    void* p = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    if (p == nullptr && PyErr_Occurred()) throw PythonError{};
    return p;
  }
  // Straight to the GPU's own function: group_rows, which makes four, takes the host 6.4 us instead of 7.1.
  static Tensor make(at::ScalarType type, at::IntArrayRef shape, const Tensor& like) {
    return at::_ops::empty_memory_format::redispatch(c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                     c10::fromIntArrayRefSlow(shape), type, at::kStrided,
                                                     like.device(), false, std::nullopt);
  }
  [[noreturn]] static void wrong_stream(long stream_dev, long dev) {
    wrong_value("stream on cuda:" + std::to_string(stream_dev) + ", operands on cuda:" + std::to_string(dev));
  }
  long long attribute(const char* name) const {
    PyObject* o = PyObject_GetAttrString(stream_, name);
    if (o == nullptr) throw PythonError{};
    const long long v = PyLong_AsLongLong(o);
    Py_DECREF(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
  }
  c10::Stream given_stream() const {
    return c10::Stream::unpack3(attribute("stream_id"), static_cast<c10::DeviceIndex>(attribute("device_index")),
                                static_cast<c10::DeviceType>(attribute("device_type")));
  }
  template <class F>
  void check(void* handle, const F& fn) {
    const auto* gpu = c10::impl::getDeviceGuardImpl(c10::DeviceType::CUDA);
    c10::OptionalDeviceGuard guard;
    if (gpu->getDevice().index() != dev_) guard.reset_device(c10::Device(c10::DeviceType::CUDA, dev_));
    int status;
    Py_BEGIN_ALLOW_THREADS status = fn(handle);
    Py_END_ALLOW_THREADS if (status != RD_OK) throw Status{status};
  }

  PyObject* stream_;
  int dev_ = -1;
};

PyObject* results(std::initializer_list<Tensor> ts) {
  if (ts.size() == 1) return THPVariable_Wrap(*ts.begin());
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = r == nullptr ? nullptr : THPVariable_Wrap(t);
    if (o == nullptr) {
      Py_XDECREF(r);
      throw PythonError{};
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

template <class T>
T* as(void* p) {
  return static_cast<T*>(p);
}

// ---------------------------------------------------------------- routing and rows

// logits, top_k, bias, score, groups, top_groups, renormalize, scale, limit, weights, ids, stream
PyObject* route(PyObject* const* a) {
  Call c(a[11]);
  const at::ScalarType type = float_type(a[0], "logits");
  const Tensor& x = need(a[0], "logits", type, 2);
  const int64_t tokens = x.size(0), experts = x.size(1);
  const int32_t top_k = integer32(a[1], "top_k"), score = integer32(a[3], "score"), groups = integer32(a[4], "groups"),
                top_groups = integer32(a[5], "top_groups"), renormalize = integer32(a[6], "renormalize");
  const float scale = real(a[7]);
  in_range(top_k, experts, RD_MAX_TOP_K);
  const void* xp = c.at(x);
  const int32_t* limit = c.scalar(a[8], "limit");
  const float* bias = none(a[2]) ? nullptr : as<float>(c.at(given(a[2], "bias", at::kFloat, {experts})));
  const Tensor weights = c.out(a[9], "weights", at::kFloat, {tokens, top_k}, x);
  const Tensor ids = c.out(a[10], "ids", at::kInt, {tokens, top_k}, x);
  float* w = as<float>(c.at(weights));
  int32_t* i = as<int32_t>(c.at(ids));
  c.launch([&](void* s) {
    return rd_route(xp, rd_type(type), bias, limit, w, i, tokens, experts, top_k, score, groups, top_groups,
                    renormalize, scale, s);
  });
  return results({weights, ids});
}

// logits, ids, d_weights, score, renormalize, scale, out, stream
PyObject* route_bwd(PyObject* const* a) {
  Call c(a[7]);
  const at::ScalarType type = float_type(a[0], "logits");
  const Tensor &x = need(a[0], "logits", type, 2), &ids = need(a[1], "ids", at::kInt, 2);
  const int64_t tokens = x.size(0), experts = x.size(1), top_k = ids.size(1);
  if (ids.size(0) != tokens) wrong_value("logits and ids must have the same rows");
  const Tensor& d = given(a[2], "d_weights", at::kFloat, {tokens, top_k});
  const int32_t score = integer32(a[3], "score"), renormalize = integer32(a[4], "renormalize");
  const float scale = real(a[5]);
  const Tensor out = c.out(a[6], "out", type, {tokens, experts}, x);
  const void* xp = c.at(x);
  const int32_t* ip = as<int32_t>(c.at(ids));
  const float* dp = as<float>(c.at(d));
  void* op = c.at(out);
  c.launch([&](void* s) {
    return rd_route_bwd(xp, rd_type(type), ip, dp, op, tokens, experts, top_k, score, renormalize, scale, s);
  });
  return results({out});
}

// ids, experts, workspace, stream
PyObject* group_rows(PyObject* const* a) {
  Call c(a[3]);
  const Tensor& ids = need(a[0], "ids", at::kInt);
  const int32_t experts = integer32(a[1], "experts");
  in_range(experts, INT32_MAX, RD_MAX_GROUPS);
  const int64_t n = ids.numel(), bytes = static_cast<int64_t>(rd_group_rows_workspace_size(n, experts));
  Tensor workspace;
  if (!none(a[2]))
    workspace = need(a[2], "workspace", at::kByte, 1);
  else if (bytes > 0)
    workspace = c.out(Py_None, "workspace", at::kByte, {bytes}, ids);
  const Tensor sizes = c.out(Py_None, "sizes", at::kInt, {experts}, ids),
               rows = c.out(Py_None, "rows", at::kInt, {n}, ids),
               slots = c.out(Py_None, "slots", at::kInt, ids.sizes(), ids),
               total = c.out(Py_None, "total", at::kInt, {1}, ids);
  const int32_t* ip = as<int32_t>(c.at(ids));
  int32_t *sp = as<int32_t>(c.at(sizes)), *rp = as<int32_t>(c.at(rows)), *lp = as<int32_t>(c.at(slots)),
          *tp = as<int32_t>(c.at(total));
  void* wp = workspace.defined() ? c.at(workspace) : nullptr;
  const size_t have = workspace.defined() ? static_cast<size_t>(workspace.numel()) : 0;
  c.launch([&](void* s) { return rd_group_rows(ip, n, experts, sp, rp, lp, tp, wp, have, s); });
  return results({sizes, rows, slots, total});
}

const Tensor& slots_of(PyObject* o, int64_t tokens) {
  const Tensor& t = need(o, "slots", at::kInt, 2);
  if (t.size(0) != tokens) wrong_value("slots must have a row for every token");
  return t;
}

// x, slots, out, stream
PyObject* dispatch_rows(PyObject* const* a) {
  Call c(a[3]);
  const Tensor& x = need(a[0], "x", at::kBFloat16, 2);
  const int64_t tokens = x.size(0), hidden = x.size(1);
  const Tensor& slots = slots_of(a[1], tokens);
  const int64_t top_k = slots.size(1);
  const Tensor out = none(a[2]) ? c.out(a[2], "out", at::kBFloat16, {tokens * top_k, hidden}, x)
                                : need(a[2], "out", at::kBFloat16, 2);
  if (out.size(1) != hidden) wrong_value("x and out must have the same width");
  const void* xp = c.at(x);
  const int32_t* sp = as<int32_t>(c.at(slots));
  void* op = c.at(out);
  const int64_t rows = out.size(0);
  c.launch([&](void* s) { return rd_dispatch_rows(xp, sp, op, tokens, top_k, hidden, rows, s); });
  return results({out});
}

// y, slots, weights, out, stream
PyObject* combine_rows(PyObject* const* a) {
  Call c(a[4]);
  const Tensor &y = need(a[0], "y", at::kBFloat16, 2), &slots = need(a[1], "slots", at::kInt, 2);
  const int64_t tokens = slots.size(0), top_k = slots.size(1), rows = y.size(0), hidden = y.size(1);
  const float* w = none(a[2]) ? nullptr : as<float>(c.at(given(a[2], "weights", at::kFloat, {tokens, top_k})));
  const Tensor out = c.out(a[3], "out", at::kBFloat16, {tokens, hidden}, y);
  const void* yp = c.at(y);
  const int32_t* sp = as<int32_t>(c.at(slots));
  void* op = c.at(out);
  c.launch([&](void* s) { return rd_combine_rows(yp, sp, w, op, tokens, top_k, hidden, rows, s); });
  return results({out});
}

// g, y, slots, weights, dy, dw, stream
PyObject* combine_rows_bwd(PyObject* const* a) {
  Call c(a[6]);
  const Tensor &g = need(a[0], "g", at::kBFloat16, 2), &y = need(a[1], "y", at::kBFloat16, 2);
  const int64_t tokens = g.size(0), hidden = g.size(1), rows = y.size(0);
  const Tensor& slots = slots_of(a[2], tokens);
  const int64_t top_k = slots.size(1);
  if (y.size(1) != hidden) wrong_value("g and y must have the same width");
  const Tensor& weights = given(a[3], "weights", at::kFloat, {tokens, top_k});
  const Tensor dy = c.out(a[4], "dy", at::kBFloat16, y.sizes(), y),
               dw = c.out(a[5], "dw", at::kFloat, {tokens, top_k}, g);
  const void *gp = c.at(g), *yp = c.at(y);
  const int32_t* sp = as<int32_t>(c.at(slots));
  const float* wp = as<float>(c.at(weights));
  void* dyp = c.at(dy);
  float* dwp = as<float>(c.at(dw));
  c.launch([&](void* s) { return rd_combine_rows_bwd(gp, yp, sp, wp, dyp, dwp, tokens, top_k, hidden, rows, s); });
  return results({dy, dw});
}

// ---------------------------------------------------------------- MX

constexpr int64_t kBlock = 32;

// A shape with its last dim replaced.
at::DimVector with_last(const Tensor& t, int64_t last) {
  at::DimVector shape(t.sizes().begin(), t.sizes().end());
  shape.back() = last;
  return shape;
}

// x, bits, limit, codes, scales, stream
PyObject* quantize_mx(PyObject* const* a) {
  Call c(a[5]);
  const at::ScalarType type = float_type(a[0], "x");
  const Tensor& x = need(a[0], "x", type);
  const int32_t bits = integer32(a[1], "bits");
  if (bits != 4 && bits != 8) wrong_value("bits must be 4 or 8");
  if (x.dim() < 1 || x.size(-1) % kBlock != 0 || x.size(-1) == 0)
    wrong_value("x's last dim must be a positive multiple of 32");
  const int64_t cols = x.size(-1), rows = x.numel() / cols;
  const int32_t* limit = c.scalar(a[2], "limit");
  const Tensor codes = c.out(a[3], "codes", bits == 4 ? at::kByte : at::kFloat8_e4m3fn,
                             with_last(x, bits == 4 ? cols / 2 : cols), x),
               scales = c.out(a[4], "scales", at::kByte, with_last(x, cols / kBlock), x);
  const void* xp = c.at(x);
  void *cp = c.at(codes), *sp = c.at(scales);
  c.launch([&](void* s) { return rd_quantize_mx(xp, rd_type(type), limit, cp, sp, rows, cols, bits, s); });
  return results({codes, scales});
}

// codes, scales, limit, out_dtype's size in bytes, out, stream
PyObject* dequantize_mx(PyObject* const* a) {
  Call c(a[5]);
  const int bits = code_bits(a[0], "codes");
  const Tensor& codes = need(a[0], "codes", bits == 4 ? at::kByte : at::kFloat8_e4m3fn);
  if (codes.dim() < 1) wrong_value("codes must have at least one dim");
  const int64_t cols = codes.size(-1) * (bits == 4 ? 2 : 1);
  if (cols % kBlock != 0 || cols == 0) wrong_value("the rows must hold a positive multiple of 32 elements");
  const int32_t* limit = c.scalar(a[2], "limit");
  const Tensor& scales = given(a[1], "scales", at::kByte, with_last(codes, cols / kBlock));
  const at::ScalarType type = none(a[4]) ? (integer(a[3]) == 4 ? at::kFloat : at::kBFloat16) : float_type(a[4], "out");
  const Tensor out = c.out(a[4], "out", type, with_last(codes, cols), codes);
  const int64_t rows = out.numel() / cols;
  const void *cp = c.at(codes), *sp = c.at(scales);
  void* op = c.at(out);
  c.launch([&](void* s) { return rd_dequantize_mx(cp, sp, limit, op, rd_type(type), rows, cols, bits, s); });
  return results({out});
}

// x_codes, x_scales, w_codes, w_scales, group_sizes, group_offset, limit, out_dtype's size in bytes, out, stream
PyObject* ragged_dot_mx(PyObject* const* a) {
  Call c(a[9]);
  const int bits = code_bits(a[0], "x_codes");
  const Tensor &x = need(a[0], "x_codes", bits == 4 ? at::kByte : at::kFloat8_e4m3fn, 2),
               &w = need(a[2], "w_codes", at::kByte, 3), &sizes = need(a[4], "group_sizes", at::kInt, 1);
  const int64_t m = x.size(0), k = x.size(1) * (bits == 4 ? 2 : 1), gl = w.size(0), n = w.size(1);
  const int32_t *offset = c.scalar(a[5], "group_offset"), *limit = c.scalar(a[6], "limit");
  if (w.size(2) * 2 != k) wrong_value("contraction sizes of x and w differ");
  const Tensor &xs = given(a[1], "x_scales", at::kByte, {m, k / kBlock}),
               &ws = given(a[3], "w_scales", at::kByte, {gl, n, k / kBlock});
  const at::ScalarType type = none(a[8]) ? (integer(a[7]) == 4 ? at::kFloat : at::kBFloat16) : float_type(a[8], "out");
  const Tensor out = c.out(a[8], "out", type, {m, n}, x);
  const void *xp = c.at(x), *xsp = c.at(xs), *wp = c.at(w), *wsp = c.at(ws);
  const int32_t* gp = as<int32_t>(c.at(sizes));
  void* op = c.at(out);
  const int64_t groups = sizes.numel();
  if (groups > INT32_MAX || gl > INT32_MAX) wrong_value("too many groups");
  c.launch([&](void* s) {
    return rd_forward_mx(xp, xsp, bits, wp, wsp, gp, static_cast<int32_t>(groups), offset, static_cast<int32_t>(gl),
                         limit, op, rd_type(type), m, k, n, s);
  });
  return results({out});
}

int64_t glu_width(const Tensor& t) {
  const int64_t width = t.size(1);
  if (width % (2 * kBlock) != 0 || width == 0) wrong_value("fused width must be a positive multiple of 64");
  return width;
}

// fused, limit, act, codes, scales, stream
PyObject* glu_fwd_mx8(PyObject* const* a) {
  Call c(a[5]);
  const Tensor& fused = need(a[0], "fused", at::kBFloat16, 2);
  const int32_t* limit = c.scalar(a[1], "limit");
  const int64_t rows = fused.size(0), width = glu_width(fused), h = width / 2;
  const Tensor act = c.out(a[2], "act", at::kBFloat16, {rows, h}, fused),
               codes = c.out(a[3], "codes", at::kFloat8_e4m3fn, {rows, width}, fused),
               scales = c.out(a[4], "scales", at::kByte, {rows, width / kBlock}, fused);
  const void* fp = c.at(fused);
  void *ap = c.at(act), *cp = c.at(codes), *sp = c.at(scales);
  c.launch([&](void* s) { return rd_glu_fwd_mx8(fp, limit, ap, cp, sp, rows, h, s); });
  return results({act, codes, scales});
}

// codes, scales, d_act, limit, weights, rows, d_fused, act, dot, stream
PyObject* glu_bwd_mx8(PyObject* const* a) {
  Call c(a[9]);
  const Tensor& codes = need(a[0], "codes", at::kFloat8_e4m3fn, 2);
  const int64_t n = codes.size(0), width = glu_width(codes), h = width / 2;
  const Tensor &scales = given(a[1], "scales", at::kByte, {n, width / kBlock}),
               &d_act = given(a[2], "d_act", at::kBFloat16, {n, h});
  const int32_t* limit = c.scalar(a[3], "limit");
  const Tensor* weights = none(a[4]) ? nullptr : &need(a[4], "weights", at::kFloat, 1);
  const int32_t* rows = none(a[5]) ? nullptr : as<int32_t>(c.at(given(a[5], "rows", at::kInt, {n})));
  const Tensor d_fused = c.out(a[6], "d_fused", at::kBFloat16, {n, width}, codes),
               act = c.out(a[7], "act", at::kBFloat16, {n, h}, codes);
  const Tensor dot = none(a[8])
                         ? c.out(a[8], "dot", at::kFloat, {weights == nullptr ? n : weights->numel()}, codes)
                         : need(a[8], "dot", at::kFloat, 1);
  if (weights != nullptr && dot.numel() != weights->numel()) wrong_value("dot and weights must have the same length");
  const void *cp = c.at(codes), *sp = c.at(scales), *dp = c.at(d_act);
  const float* wp = weights == nullptr ? nullptr : as<float>(c.at(*weights));
  void *fp = c.at(d_fused), *ap = c.at(act);
  float* op = as<float>(c.at(dot));
  const int64_t slots = dot.numel();
  c.launch([&](void* s) { return rd_glu_bwd_mx8(cp, sp, dp, limit, wp, rows, fp, ap, op, n, h, slots, s); });
  return results({d_fused, act, dot});
}

// ---------------------------------------------------------------- the module

// No C++ exception leaves the module.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
  try {
    return F(args);
  } catch (const Refusal& e) {
    PyErr_SetString(e.type, e.what.c_str());
  } catch (const Status& e) {
    PyErr_SetString(g_status_error, rd_status_string(e.code));
  } catch (const PythonError&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_out_of_memory, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The exceptions for a nonzero status and for a failed allocation, and the function that gives the current
// stream's handle.
PyObject* setup(PyObject*, PyObject* const* args, Py_ssize_t n) {
  PyObject** const kept[] = {&g_status_error, &g_out_of_memory, &g_raw_stream};
  if (n != 3) return PyErr_Format(PyExc_TypeError, "expected 3 arguments, got %zd", n);
  for (int i = 0; i < 3; ++i) {
    Py_INCREF(args[i]);
    Py_XDECREF(*kept[i]);
    *kept[i] = args[i];
  }
  Py_RETURN_NONE;
}

#define RD_METHOD(fn, n) \
  {#fn, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<fn, n>)), METH_FASTCALL, nullptr}

PyMethodDef g_methods[] = {
    {"setup", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(setup)), METH_FASTCALL, nullptr},
    RD_METHOD(route, 12),
    RD_METHOD(route_bwd, 8),
    RD_METHOD(group_rows, 4),
    RD_METHOD(dispatch_rows, 4),
    RD_METHOD(combine_rows, 5),
    RD_METHOD(combine_rows_bwd, 7),
    RD_METHOD(quantize_mx, 6),
    RD_METHOD(dequantize_mx, 6),
    RD_METHOD(ragged_dot_mx, 10),
    RD_METHOD(glu_fwd_mx8, 6),
    RD_METHOD(glu_bwd_mx8, 10),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_rd", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rd() { return PyModule_Create(&g_module); }
