// torch_ops.cpp -- the torch-tensor forms of the operators around the
// products: a tensor's address, pitch and format read and checked, the
// workspace taken from torch's allocator and the current stream found, then
// one call of the C entry point.  No arithmetic.
//
// A small call's time is its host time.  Written in Python, the checks of five
// tensors and the stream cost as much as the launch (norm of one token: 9.3 us
// a call, 3 of them the launch); here they are a fraction of a microsecond.
//
// Every function returns the thl_status of its call; wrong tensors raise
// ValueError, a workspace that does not fit torch.OutOfMemoryError, and nothing
// is launched.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/Allocator.h>
#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <exception>
#include <string>

#include "../../include/thl.h"

namespace {

struct Refused : std::exception {
  char text[256];
  explicit Refused(const char* f, ...) {
    va_list ap;
    va_start(ap, f);
    vsnprintf(text, sizeof text, f, ap);
    va_end(ap);
  }
  const char* what() const noexcept override { return text; }
};
struct Raised : std::exception {};  // a Python error is set

// Where autograd records (backward or forward mode), a call that it does not
// see would be a constant to it, without a word.
const at::Tensor& tensor(const char* what, PyObject* o) {
  if (!THPVariable_Check(o)) throw Refused("%s: a torch tensor is expected", what);
  const at::Tensor& t = THPVariable_Unpack(o);
  const c10::AutogradState& mode = c10::AutogradState::get_tls_state();
  if ((mode.get_grad_mode() && t.requires_grad()) || (mode.get_fw_grad_mode() && t._fw_grad(0).defined()))
    throw Refused("%s: requires a gradient, which these calls do not record; call them under torch.no_grad() or inside "
                  "a torch.autograd.Function", what);
  return t;
}
bool given(PyObject* o) { return o != Py_None; }

int format(const char* what, const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat:
      return THL_F32;
    case at::kHalf:
      return THL_F16;
    case at::kBFloat16:
      return THL_BF16;
    case at::kChar:
    case at::kByte:
      return THL_I8;
    case at::kInt:
      return THL_I32;
    case at::kFloat8_e4m3fn:
      return THL_E4M3;
    case at::kFloat8_e5m2:
      return THL_E5M2;
    case at::kFloat8_e8m0fnu:
      return THL_E8M0;
    default:
      throw Refused("%s: no format for tensors of type %s", what, c10::toString(t.scalar_type()));
  }
}

// The first tensor of a call: its device is everyone's.
int device_of(const char* what, const at::Tensor& t) {
  if (!t.is_cuda() || t.dim() != 2) throw Refused("%s: a (tokens, features) tensor on a GPU is expected", what);
  return t.get_device();
}
void same_device(const char* what, const at::Tensor& t, int dev) {
  if (!t.is_cuda() || t.get_device() != dev) throw Refused("%s: on the others' GPU (cuda:%d) is expected", what, dev);
}

struct Mat {
  void* p = nullptr;
  int64_t ld = 0;
};
// An (n, m) tensor whose rows are contiguous, maybe pitched.
Mat tokens(const char* what, const at::Tensor& t, int dev, int64_t n, int64_t m) {
  same_device(what, t, dev);
  if (t.dim() != 2 || t.size(0) != n || t.size(1) != m)
    throw Refused("%s: a tensor of shape (%lld, %lld) is expected", what, static_cast<long long>(n),
                  static_cast<long long>(m));
  if (m > 1 && t.stride(1) != 1) throw Refused("%s: features must be contiguous", what);
  int64_t ld = t.stride(0);
  if (n <= 1 && ld < m) ld = m;
  if (n <= 1 && ld < 1) ld = 1;
  return {t.data_ptr(), ld};
}
// n rows of at least `bytes` one-byte elements.
Mat byte_rows(const char* what, const at::Tensor& t, int dev, int64_t n, int64_t bytes) {
  if (t.element_size() != 1 || t.dim() != 2 || t.size(1) < bytes)
    throw Refused("%s: rows of at least %lld bytes are expected", what, static_cast<long long>(bytes));
  return tokens(what, t, dev, n, t.size(1));
}
void* vec(const char* what, const at::Tensor& t, int dev, int64_t n) {
  same_device(what, t, dev);
  if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    throw Refused("%s: %lld contiguous elements are expected", what, static_cast<long long>(n));
  return t.data_ptr();
}
void* table(const char* what, const at::Tensor& t, int dev, int64_t n, int64_t m, at::ScalarType type) {
  same_device(what, t, dev);
  if (t.dim() != 2 || t.size(0) != n || t.size(1) != m || !t.is_contiguous() || t.scalar_type() != type)
    throw Refused("%s: a contiguous (%lld, %lld) tensor of %s is expected", what, static_cast<long long>(n),
                  static_cast<long long>(m), c10::toString(type));
  return t.data_ptr();
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return static_cast<float>(v);
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}
const char* text(PyObject* o) {
  const char* s = PyUnicode_AsUTF8(o);
  if (!s) throw Raised();
  return s;
}

// A launch's device, stream and workspace.  The workspace goes back to
// torch's allocator, which hands it on in the order of the stream it was
// taken on: the current one, which is the launch's.
struct Launch {
  c10::DeviceGuard guard;
  struct ihipStream_t* stream;
  c10::DataPtr workspace;
  explicit Launch(int dev)
      : guard(c10::Device(c10::DeviceType::CUDA, static_cast<c10::DeviceIndex>(dev))),
        stream(c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(dev)).stream()) {}
  void* take(size_t bytes) {
    if (bytes == 0) return nullptr;
    workspace = c10::GetAllocator(c10::DeviceType::CUDA)->allocate(bytes);
    return workspace.get();
  }
};

// x, w, y, eps, residual, residual_out, scale, sf
thl_status rmsnorm(PyObject* const* a) {
  const at::Tensor &x = tensor("x", a[0]), &w = tensor("w", a[1]), &y = tensor("y", a[2]);
  const int dev = device_of("x", x);
  const int64_t n = x.size(0), m = x.size(1);
  const Mat mx = tokens("x", x, dev, n, m);
  const bool fp4 = y.scalar_type() == at::kByte;
  Mat my = tokens("y", y, dev, n, fp4 ? (m + 1) / 2 : m), mr, ms, mf;
  if (fp4) my.ld *= 2;
  thl_norm_types ty = {static_cast<thl_dtype>(format("x", x)), THL_NONE, static_cast<thl_dtype>(format("w", w)),
                       fp4 ? THL_E2M1X2 : static_cast<thl_dtype>(format("y", y))};
  const void* pw = vec("w", w, dev, m);
  if (given(a[4])) {
    const at::Tensor& r = tensor("residual", a[4]);
    mr = tokens("residual", r, dev, n, m);
    ty.r = static_cast<thl_dtype>(format("residual", r));
  }
  if (given(a[5])) {
    const at::Tensor& s = tensor("residual_out", a[5]);
    if (!given(a[4]) || format("residual_out", s) != ty.r)
      throw Refused("residual_out: with a residual, of its type");
    ms = tokens("residual_out", s, dev, n, m);
  }
  if (given(a[7])) mf = byte_rows("sf", tensor("sf", a[7]), dev, n, (m + 31) / 32);
  const float eps = number(a[3]), scale = number(a[6]);
  Launch l(dev);
  return thl_rmsnorm(m, n, mx.p, mx.ld, mr.p, mr.ld, ms.p, ms.ld, pw, eps, scale, my.p, my.ld,
                     static_cast<uint8_t*>(mf.p), mf.ld, &ty, l.stream);
}

// s, dy, w, dx, dw, eps, dres
thl_status rmsnorm_backward(PyObject* const* a) {
  const at::Tensor &s = tensor("s", a[0]), &dy = tensor("dy", a[1]), &w = tensor("w", a[2]), &dx = tensor("dx", a[3]);
  const int dev = device_of("s", s);
  const int64_t n = s.size(0), m = s.size(1);
  const Mat ms = tokens("s", s, dev, n, m), mg = tokens("dy", dy, dev, n, m), mx = tokens("dx", dx, dev, n, m);
  thl_norm_grad_types ty = {static_cast<thl_dtype>(format("s", s)), static_cast<thl_dtype>(format("w", w)),
                            static_cast<thl_dtype>(format("dy", dy)), THL_NONE};
  const void* pw = vec("w", w, dev, m);
  Mat mr;
  if (format("dx", dx) != ty.g) throw Refused("dx: dy's type is expected");
  if (given(a[6])) {
    const at::Tensor& r = tensor("dres", a[6]);
    if (format("dres", r) != ty.g) throw Refused("dres: dy's type is expected");
    mr = tokens("dres", r, dev, n, m);
  }
  void* pd = nullptr;
  if (given(a[4])) {
    const at::Tensor& d = tensor("dw", a[4]);
    pd = vec("dw", d, dev, m);
    ty.dw = static_cast<thl_dtype>(format("dw", d));
  }
  const float eps = number(a[5]);
  Launch l(dev);
  const size_t need = pd ? thl_rmsnorm_backward_workspace(m, n) : 0;
  void* ws = l.take(need);
  return thl_rmsnorm_backward(m, n, ms.p, ms.ld, mg.p, mg.ld, mr.p, mr.ld, pw, eps, mx.p, mx.ld, pd, ws, need, &ty,
                              l.stream);
}

// x, w, b, y, eps, residual, residual_out, scale, sf
thl_status layernorm(PyObject* const* a) {
  const at::Tensor &x = tensor("x", a[0]), &y = tensor("y", a[3]);
  const int dev = device_of("x", x);
  const int64_t n = x.size(0), m = x.size(1);
  const Mat mx = tokens("x", x, dev, n, m);
  const bool fp4 = y.scalar_type() == at::kByte;
  Mat my = tokens("y", y, dev, n, fp4 ? (m + 1) / 2 : m), mr, ms, mf;
  if (fp4) my.ld *= 2;
  thl_norm_types ty = {static_cast<thl_dtype>(format("x", x)), THL_NONE, THL_NONE,
                       fp4 ? THL_E2M1X2 : static_cast<thl_dtype>(format("y", y))};
  void *pw = nullptr, *pb = nullptr;
  if (given(a[1])) {
    const at::Tensor& w = tensor("w", a[1]);
    pw = vec("w", w, dev, m);
    ty.w = static_cast<thl_dtype>(format("w", w));
  }
  if (given(a[2])) {
    const at::Tensor& b = tensor("b", a[2]);
    pb = vec("b", b, dev, m);
    if (pw && format("b", b) != ty.w) throw Refused("b: w's type is expected");
    ty.w = static_cast<thl_dtype>(format("b", b));
  }
  if (given(a[5])) {
    const at::Tensor& r = tensor("residual", a[5]);
    mr = tokens("residual", r, dev, n, m);
    ty.r = static_cast<thl_dtype>(format("residual", r));
  }
  if (given(a[6])) {
    const at::Tensor& s = tensor("residual_out", a[6]);
    if (!given(a[5]) || format("residual_out", s) != ty.r)
      throw Refused("residual_out: with a residual, of its type");
    ms = tokens("residual_out", s, dev, n, m);
  }
  if (given(a[8])) mf = byte_rows("sf", tensor("sf", a[8]), dev, n, (m + 31) / 32);
  const float eps = number(a[4]), scale = number(a[7]);
  Launch l(dev);
  return thl_layernorm(m, n, mx.p, mx.ld, mr.p, mr.ld, ms.p, ms.ld, pw, pb, eps, scale, my.p, my.ld,
                       static_cast<uint8_t*>(mf.p), mf.ld, &ty, l.stream);
}

// s, dy, w, dx, dw, db, eps, dres
thl_status layernorm_backward(PyObject* const* a) {
  const at::Tensor &s = tensor("s", a[0]), &dy = tensor("dy", a[1]), &dx = tensor("dx", a[3]);
  const int dev = device_of("s", s);
  const int64_t n = s.size(0), m = s.size(1);
  const Mat ms = tokens("s", s, dev, n, m), mg = tokens("dy", dy, dev, n, m), mx = tokens("dx", dx, dev, n, m);
  thl_norm_grad_types ty = {static_cast<thl_dtype>(format("s", s)), THL_NONE, static_cast<thl_dtype>(format("dy", dy)),
                            THL_NONE};
  void *pw = nullptr, *pd = nullptr, *pe = nullptr;
  Mat mr;
  if (given(a[2])) {
    const at::Tensor& w = tensor("w", a[2]);
    pw = vec("w", w, dev, m);
    ty.w = static_cast<thl_dtype>(format("w", w));
  }
  if (format("dx", dx) != ty.g) throw Refused("dx: dy's type is expected");
  if (given(a[7])) {
    const at::Tensor& r = tensor("dres", a[7]);
    if (format("dres", r) != ty.g) throw Refused("dres: dy's type is expected");
    mr = tokens("dres", r, dev, n, m);
  }
  if (given(a[4])) {
    const at::Tensor& d = tensor("dw", a[4]);
    pd = vec("dw", d, dev, m);
    ty.dw = static_cast<thl_dtype>(format("dw", d));
  }
  if (given(a[5])) {
    const at::Tensor& d = tensor("db", a[5]);
    pe = vec("db", d, dev, m);
    if (pd && format("db", d) != ty.dw) throw Refused("db: dw's type is expected");
    ty.dw = static_cast<thl_dtype>(format("db", d));
  }
  const float eps = number(a[6]);
  Launch l(dev);
  const size_t need = pd || pe ? thl_layernorm_backward_workspace(m, n) : 0;
  void* ws = l.take(need);
  return thl_layernorm_backward(m, n, ms.p, ms.ld, mg.p, mg.ld, mr.p, mr.ld, pw, eps, mx.p, mx.ld, pd, pe, ws, need,
                                &ty, l.stream);
}

// x, y, sf, y_t, sf_t
thl_status mx_quantize(PyObject* const* a) {
  const at::Tensor& x = tensor("x", a[0]);
  const int dev = device_of("x", x);
  const int64_t n = x.size(0), m = x.size(1);
  const Mat mx = tokens("x", x, dev, n, m);
  Mat out[2], sf[2];
  int type = THL_NONE;
  if (given(a[1]) != given(a[2])) throw Refused("y and sf go together");
  if (given(a[3]) != given(a[4])) throw Refused("y_t and sf_t go together");
  static const char* const names[2][2] = {{"y", "sf"}, {"y_t", "sf_t"}};
  for (int i = 0; i < 2; ++i) {
    if (!given(a[1 + 2 * i])) continue;
    const at::Tensor& y = tensor(names[i][0], a[1 + 2 * i]);
    const bool fp4 = y.scalar_type() == at::kByte;
    const int kind = fp4 ? THL_E2M1X2 : format(names[i][0], y);
    if (type != THL_NONE && kind != type) throw Refused("y_t: y's type is expected");
    type = kind;
    const int64_t rows = i ? m : n, cols = i ? n : m;
    out[i] = tokens(names[i][0], y, dev, rows, fp4 ? (cols + 1) / 2 : cols);
    if (fp4) out[i].ld *= 2;
    sf[i] = byte_rows(names[i][1], tensor(names[i][1], a[2 + 2 * i]), dev, rows, (cols + 31) / 32);
  }
  if (type == THL_NONE) throw Refused("y with sf, or y_t with sf_t, is expected");
  const int type_x = format("x", x);
  Launch l(dev);
  return thl_mx_quantize(m, n, mx.p, mx.ld, out[0].p, out[0].ld, static_cast<uint8_t*>(sf[0].p), sf[0].ld, out[1].p,
                         out[1].ld, static_cast<uint8_t*>(sf[1].p), sf[1].ld, static_cast<thl_dtype>(type_x),
                         static_cast<thl_dtype>(type), l.stream);
}

thl_route router(const at::Tensor& logits, PyObject* score, PyObject* renormalize, PyObject* scale) {
  thl_route how{};
  how.type = static_cast<thl_dtype>(format("logits", logits));
  const char* s = text(score);
  if (strcmp(s, "sigmoid") == 0)
    how.score = THL_ROUTE_SIGMOID;
  else if (strcmp(s, "softmax") != 0)
    throw Refused("score: softmax or sigmoid is expected");
  how.renormalize = truth(renormalize);
  how.scale = number(scale);
  return how;
}

// logits, ids, weights, score, renormalize, scale, bias
thl_status moe_route(PyObject* const* a) {
  const at::Tensor &logits = tensor("logits", a[0]), &ids = tensor("ids", a[1]);
  const int dev = device_of("logits", logits);
  const int64_t n = logits.size(0), experts = logits.size(1);
  if (ids.dim() != 2) throw Refused("ids: (tokens, choices) is expected");
  const int64_t topk = ids.size(1);
  const Mat ml = tokens("logits", logits, dev, n, experts);
  int32_t* pi = static_cast<int32_t*>(table("ids", ids, dev, n, topk, at::kInt));
  float* pw = static_cast<float*>(table("weights", tensor("weights", a[2]), dev, n, topk, at::kFloat));
  const thl_route how = router(logits, a[3], a[4], a[5]);
  const float* pb = nullptr;
  if (given(a[6])) {
    const at::Tensor& b = tensor("bias", a[6]);
    pb = static_cast<const float*>(vec("bias", b, dev, experts));
    if (b.scalar_type() != at::kFloat) throw Refused("bias: float32 is expected");
  }
  Launch l(dev);
  return thl_moe_route(n, topk, experts, ml.p, ml.ld, pb, &how, pi, pw, l.stream);
}

// logits, ids, dweights, dlogits, score, renormalize, scale
thl_status moe_route_backward(PyObject* const* a) {
  const at::Tensor &logits = tensor("logits", a[0]), &ids = tensor("ids", a[1]), &dl = tensor("dlogits", a[3]);
  const int dev = device_of("logits", logits);
  const int64_t n = logits.size(0), experts = logits.size(1);
  if (ids.dim() != 2) throw Refused("ids: (tokens, choices) is expected");
  const int64_t topk = ids.size(1);
  const Mat ml = tokens("logits", logits, dev, n, experts), md = tokens("dlogits", dl, dev, n, experts);
  if (dl.scalar_type() != logits.scalar_type()) throw Refused("dlogits: the logits' type is expected");
  const int32_t* pi = static_cast<int32_t*>(table("ids", ids, dev, n, topk, at::kInt));
  const float* pw = static_cast<float*>(table("dweights", tensor("dweights", a[2]), dev, n, topk, at::kFloat));
  const thl_route how = router(logits, a[4], a[5], a[6]);
  Launch l(dev);
  return thl_moe_route_backward(n, topk, experts, ml.p, ml.ld, &how, pi, pw, md.p, md.ld, l.stream);
}

// An (experts, rows, k) tensor of weights with its scales and bias.
thl_expert_matrix experts_of(const char* what, const at::Tensor& w, int dev, int64_t experts, int64_t rows, int64_t k,
                             const char* what_sf, PyObject* sf, const char* what_b, PyObject* bias) {
  thl_expert_matrix o{};
  same_device(what, w, dev);
  const bool fp4 = w.scalar_type() == at::kByte;
  const int64_t cols = fp4 ? (k + 1) / 2 : k;
  if (w.dim() != 3 || w.size(0) != experts || w.size(1) != rows || w.size(2) != cols)
    throw Refused("%s: a tensor of shape (%lld, %lld, %lld) is expected", what, static_cast<long long>(experts),
                  static_cast<long long>(rows), static_cast<long long>(cols));
  if (cols > 1 && w.stride(2) != 1) throw Refused("%s: rows must be contiguous", what);
  const int64_t packed = fp4 ? 2 : 1;
  o.w = w.data_ptr();
  o.ld = packed * (rows > 1 ? w.stride(1) : cols), o.stride = packed * (experts > 1 ? w.stride(0) : 0);
  o.type = fp4 ? THL_E2M1X2 : static_cast<thl_dtype>(format(what, w));
  o.type_bias = THL_NONE;
  if (given(sf)) {
    const at::Tensor& s = tensor(what_sf, sf);
    same_device(what_sf, s, dev);
    const int64_t blocks = (k + 31) / 32;
    if (s.element_size() != 1 || s.dim() != 3 || s.size(0) != experts || s.size(1) != rows || s.size(2) < blocks ||
        (blocks > 1 && s.stride(2) != 1))
      throw Refused("%s: (%lld, %lld) rows of at least %lld bytes are expected", what_sf,
                    static_cast<long long>(experts), static_cast<long long>(rows), static_cast<long long>(blocks));
    o.sf = static_cast<const uint8_t*>(s.data_ptr());
    o.ld_sf = rows > 1 ? s.stride(1) : blocks, o.stride_sf = experts > 1 ? s.stride(0) : 0;
  }
  if (given(bias)) {
    const at::Tensor& b = tensor(what_b, bias);
    same_device(what_b, b, dev);
    if (b.dim() != 2 || b.size(0) != experts || b.size(1) != rows || (rows > 1 && b.stride(1) != 1))
      throw Refused("%s: (%lld, %lld) values are expected", what_b, static_cast<long long>(experts),
                    static_cast<long long>(rows));
    o.bias = b.data_ptr(), o.stride_bias = experts > 1 ? b.stride(0) : 0;
    o.type_bias = static_cast<thl_dtype>(format(what_b, b));
  }
  return o;
}

// x, ids, weights, w1, w2, y, gated, act, sf1, sf2, b1, b2
thl_status moe_layer(PyObject* const* a) {
  const at::Tensor &x = tensor("x", a[0]), &ids = tensor("ids", a[1]), &w1 = tensor("w1", a[3]),
                   &w2 = tensor("w2", a[4]), &y = tensor("y", a[5]);
  const int dev = device_of("x", x);
  const int64_t n = x.size(0), m = x.size(1);
  if (ids.dim() != 2 || (ids.scalar_type() != at::kInt && ids.scalar_type() != at::kLong))
    throw Refused("ids: (tokens, choices) of int32 or int64 is expected");
  const int64_t topk = ids.size(1);
  const Mat mx = tokens("x", x, dev, n, m), my = tokens("y", y, dev, n, m), mi = tokens("ids", ids, dev, n, topk);
  const float* pw = static_cast<float*>(table("weights", tensor("weights", a[2]), dev, n, topk, at::kFloat));
  const bool gated = truth(a[6]);
  if (w1.dim() != 3 || (gated && w1.size(1) % 2 != 0)) throw Refused("w1: (experts, rows, features) is expected");
  const int64_t experts = w1.size(0), hidden = gated ? w1.size(1) / 2 : w1.size(1);
  unsigned flags = gated ? THL_MOE_GATED : 0;
  const char* act = text(a[7]);
  if (strcmp(act, "relu") == 0)
    flags |= THL_MOE_RELU;
  else if (strcmp(act, "gelu") == 0)
    flags |= THL_MOE_GELU;
  else if (strcmp(act, "silu") == 0)
    flags |= THL_MOE_SILU;
  else if (strcmp(act, "none") != 0)
    throw Refused("act: none, relu, gelu or silu is expected");
  const thl_expert_matrix up = experts_of("w1", w1, dev, experts, w1.size(1), m, "sf1", a[8], "b1", a[10]);
  const thl_expert_matrix down = experts_of("w2", w2, dev, experts, m, hidden, "sf2", a[9], "b2", a[11]);
  const thl_dtype type_x = static_cast<thl_dtype>(format("x", x)), type_y = static_cast<thl_dtype>(format("y", y));
  Launch l(dev);
  const size_t need = thl_moe_layer_workspace(m, hidden, n, topk);
  void* ws = l.take(need);
  return thl_moe_layer(m, hidden, n, topk, experts, mx.p, mx.ld, mi.p, mi.ld, static_cast<int>(ids.element_size()), pw,
                       &up, &down, flags, my.p, my.ld, type_x, type_y, ws, need, l.stream);
}

// ids, experts, rows, offsets, order
thl_status moe_sort(PyObject* const* a) {
  const at::Tensor& ids = tensor("ids", a[0]);
  const int dev = device_of("ids", ids);
  const int64_t n = ids.size(0), topk = ids.size(1), experts = integer(a[1]);
  if (ids.scalar_type() != at::kInt && ids.scalar_type() != at::kLong) throw Refused("ids: int32 or int64 is expected");
  const Mat mi = tokens("ids", ids, dev, n, topk);
  int32_t* rows = static_cast<int32_t*>(table("rows", tensor("rows", a[2]), dev, n, topk, at::kInt));
  const at::Tensor& off = tensor("offsets", a[3]);
  int32_t* offsets = static_cast<int32_t*>(vec("offsets", off, dev, experts + 1));
  int32_t* order = nullptr;
  if (off.scalar_type() != at::kInt) throw Refused("offsets: int32 is expected");
  if (given(a[4])) {
    const at::Tensor& o = tensor("order", a[4]);
    order = static_cast<int32_t*>(vec("order", o, dev, n * topk));
    if (o.scalar_type() != at::kInt) throw Refused("order: int32 is expected");
  }
  Launch l(dev);
  const size_t need = thl_moe_sort_workspace(n, topk, experts);
  void* ws = l.take(need);
  return thl_moe_sort(n, topk, experts, mi.p, mi.ld, static_cast<int>(ids.element_size()), rows, offsets, order, ws,
                      need, l.stream);
}

// (n, choices) places: their address and the choices.
const int32_t* choices(PyObject* o, int dev, int64_t n, int64_t* topk) {
  const at::Tensor& r = tensor("rows", o);
  if (r.dim() != 2) throw Refused("rows: (tokens, choices) is expected");
  *topk = r.size(1);
  return static_cast<const int32_t*>(table("rows", r, dev, n, *topk, at::kInt));
}

// x, rows, y, sf, sf_y, type_x
thl_status moe_gather(PyObject* const* a) {
  const at::Tensor &x = tensor("x", a[0]), &y = tensor("y", a[2]);
  const int dev = device_of("x", x);
  const int64_t n = x.size(0), cols = x.size(1);
  int64_t topk = 0, packed = 1;
  const int32_t* rows = choices(a[1], dev, n, &topk);
  const Mat mx = tokens("x", x, dev, n, cols);
  if (y.dim() != 2 || y.scalar_type() != x.scalar_type()) throw Refused("y: a (rows, features) tensor of x's type");
  const int64_t rows_y = y.size(0);
  const Mat my = tokens("y", y, dev, rows_y, cols);
  int type = format("x", x);
  if (given(a[5])) {
    static const struct {
      const char* name;
      int type, packed;
    } kinds[] = {{"e2m1", THL_E2M1X2, 2}, {"i4", THL_I4X2, 2}, {"u4", THL_U4X2, 2},
                 {"e4m3", THL_E4M3, 1},   {"e5m2", THL_E5M2, 1}, {"i8", THL_I8, 1}};
    const char* want = text(a[5]);
    bool found = false;
    for (const auto& k : kinds)
      if (x.element_size() == 1 && strcmp(k.name, want) == 0) type = k.type, packed = k.packed, found = true;
    if (!found) throw Refused("type_x: an 8- or 4-bit format of a one-byte tensor is expected");
  }
  const int64_t m = packed * cols;
  Mat mf, mg;
  if (given(a[3]) != given(a[4])) throw Refused("sf and sf_y go together");
  if (given(a[3])) {
    mf = byte_rows("sf", tensor("sf", a[3]), dev, n, (m + 31) / 32);
    mg = byte_rows("sf_y", tensor("sf_y", a[4]), dev, rows_y, (m + 31) / 32);
  }
  Launch l(dev);
  return thl_moe_gather(m, n, topk, mx.p, packed * mx.ld, static_cast<const uint8_t*>(mf.p), mf.ld, rows, rows_y, my.p,
                        packed * my.ld, static_cast<uint8_t*>(mg.p), mg.ld, static_cast<thl_dtype>(type), l.stream);
}

// x, rows, y, weights
thl_status moe_combine(PyObject* const* a) {
  const at::Tensor &x = tensor("x", a[0]), &y = tensor("y", a[2]);
  const int dev = device_of("x", x);
  device_of("y", y);
  const int64_t rows_x = x.size(0), m = x.size(1), n = y.size(0);
  int64_t topk = 0;
  const int32_t* rows = choices(a[1], dev, n, &topk);
  const Mat mx = tokens("x", x, dev, rows_x, m), my = tokens("y", y, dev, n, m);
  const float* weights =
      given(a[3]) ? static_cast<float*>(table("weights", tensor("weights", a[3]), dev, n, topk, at::kFloat)) : nullptr;
  Launch l(dev);
  return thl_moe_combine(m, n, topk, mx.p, mx.ld, rows_x, rows, weights, my.p, my.ld,
                         static_cast<thl_dtype>(format("x", x)), static_cast<thl_dtype>(format("y", y)), l.stream);
}

// dy, x, rows, weights, dx, dweights
thl_status moe_combine_backward(PyObject* const* a) {
  const at::Tensor& dy = tensor("dy", a[0]);
  const int dev = device_of("dy", dy);
  if ((!given(a[1]) && !given(a[4])) || (given(a[5]) && !given(a[1])))
    throw Refused("x is needed for dweights, x or dx for the rows");
  const at::Tensor& like = given(a[1]) ? tensor("x", a[1]) : tensor("dx", a[4]);
  device_of("x", like);
  const int64_t n = dy.size(0), m = dy.size(1), rows_x = like.size(0);
  int64_t topk = 0;
  const int32_t* rows = choices(a[2], dev, n, &topk);
  const Mat mg = tokens("dy", dy, dev, n, m);
  Mat mx, md;
  float *weights = nullptr, *dweights = nullptr;
  if (given(a[1])) mx = tokens("x", like, dev, rows_x, m);
  if (given(a[4])) {
    const at::Tensor& dx = tensor("dx", a[4]);
    if (dx.scalar_type() != like.scalar_type()) throw Refused("dx: x's type is expected");
    md = tokens("dx", dx, dev, rows_x, m);
    weights = static_cast<float*>(table("weights", tensor("weights", a[3]), dev, n, topk, at::kFloat));
  }
  if (given(a[5]))
    dweights = static_cast<float*>(table("dweights", tensor("dweights", a[5]), dev, n, topk, at::kFloat));
  Launch l(dev);
  return thl_moe_combine_backward(m, n, topk, mg.p, mg.ld, mx.p, mx.ld, rows_x, rows, weights, md.p, md.ld, dweights,
                                  static_cast<thl_dtype>(format("dy", dy)), static_cast<thl_dtype>(format("x", like)),
                                  l.stream);
}

// w, x, d, scales, group, type_w, zeros, c, alpha, beta, bias, act
thl_status gemm_w4(PyObject* const* a) {
  const at::Tensor &w = tensor("w", a[0]), &x = tensor("x", a[1]), &d = tensor("d", a[2]),
                   &scales = tensor("scales", a[3]);
  const int dev = device_of("x", x);
  const int64_t n = x.size(0), k = x.size(1), m = w.dim() == 2 ? w.size(0) : -1, group = integer(a[4]);
  const char *type_w = text(a[5]), *act = text(a[11]);
  thl_dtypes dt = {THL_U4X2, static_cast<thl_dtype>(format("x", x)), THL_NONE, static_cast<thl_dtype>(format("d", d)),
                   THL_NONE, THL_F32};
  if (strcmp(type_w, "e2m1") == 0)
    dt.a = THL_E2M1X2;
  else if (strcmp(type_w, "i4") == 0)
    dt.a = THL_I4X2;
  else if (strcmp(type_w, "u4") != 0)
    throw Refused("type_w: u4, i4 or e2m1 is expected");
  if (w.element_size() != 1 || group < 1) throw Refused("w: two codes a byte, in groups of a positive length");
  const Mat mw = tokens("w", w, dev, m, (k + 1) / 2), mx = tokens("x", x, dev, n, k), md = tokens("d", d, dev, n, m);
  const int64_t groups = k == 0 ? 0 : (k - 1) / group + 1;
  thl_group_scales gs{};
  gs.group = group;
  Mat ms;
  if (dt.a == THL_E2M1X2) {
    ms = byte_rows("scales", scales, dev, m, groups);
    gs.type = THL_E8M0;
  } else {
    ms = tokens("scales", scales, dev, m, groups);
    gs.type = static_cast<thl_dtype>(format("scales", scales));
  }
  gs.scales = ms.p, gs.ld_scales = ms.ld;
  if (given(a[6])) {
    const Mat mz = byte_rows("zeros", tensor("zeros", a[6]), dev, m, groups);
    gs.zeros = static_cast<const uint8_t*>(mz.p), gs.ld_zeros = mz.ld;
  }
  const float alpha = number(a[8]), beta = number(a[9]);
  Mat mc;
  if (beta != 0.0f) {
    if (!given(a[7])) throw Refused("beta without c");
    const at::Tensor& c = tensor("c", a[7]);
    mc = tokens("c", c, dev, n, m);
    dt.c = static_cast<thl_dtype>(format("c", c));
  }
  thl_epilogue epi{};
  if (strcmp(act, "relu") == 0)
    epi.flags = THL_EPI_RELU;
  else if (strcmp(act, "gelu") == 0)
    epi.flags = THL_EPI_GELU;
  else if (strcmp(act, "none") != 0)
    throw Refused("act: none, relu or gelu is expected");
  if (given(a[10])) {
    const at::Tensor& b = tensor("bias", a[10]);
    epi.flags |= THL_EPI_BIAS;
    epi.bias = vec("bias", b, dev, m);
    dt.bias = static_cast<thl_dtype>(format("bias", b));
  }
  Launch l(dev);
  const size_t need = thl_gemm_w4_workspace(m, n, k);
  void* ws = l.take(need);
  return thl_gemm_w4(m, n, k, mw.p, 2 * mw.ld, &gs, mx.p, mx.ld, mc.p, mc.ld, md.p, md.ld, alpha, beta, &dt, &epi, ws,
                     need, l.stream);
}

// torch.OutOfMemoryError, which programs catch to go on with less (torch does
// not export its C++ handle).
void out_of_memory(const char* what) {
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
  if (type) PyErr_SetString(type, what);
  Py_XDECREF(type);
  Py_XDECREF(torch);
}

// An output was written: torch's own in-place operations count that, so that
// autograd notices when a tensor that it keeps for a backward has changed.
// (Inference tensors have no counter.)
void written(PyObject* o) {
  if (!given(o)) return;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// One Python function: N positional arguments, of which those at OUT are
// outputs; errors as exceptions.
template <thl_status (*F)(PyObject* const*), Py_ssize_t N, int... OUT>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n != N) throw Refused("%d arguments are expected", static_cast<int>(N));
    const thl_status status = F(args);
    // (a HIP error may come behind a first launch)
    if (status == THL_OK || status == THL_ERR_HIP) (written(args[OUT]), ...);
    return PyLong_FromLong(status);
  } catch (const Raised&) {
    return nullptr;
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    out_of_memory(e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <thl_status (*F)(PyObject* const*), Py_ssize_t N, int... OUT>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N, OUT...>)), METH_FASTCALL,
          nullptr};
}

PyMethodDef methods[] = {
    method<rmsnorm, 8, 2, 5, 7>("rmsnorm"),
    method<rmsnorm_backward, 7, 3, 4>("rmsnorm_backward"),
    method<layernorm, 9, 3, 6, 8>("layernorm"),
    method<layernorm_backward, 8, 3, 4, 5>("layernorm_backward"),
    method<mx_quantize, 5, 1, 2, 3, 4>("mx_quantize"),
    method<moe_route, 7, 1, 2>("moe_route"),
    method<moe_route_backward, 7, 3>("moe_route_backward"),
    method<moe_layer, 12, 5>("moe_layer"),
    method<moe_sort, 5, 2, 3, 4>("moe_sort"),
    method<moe_gather, 6, 2, 4>("moe_gather"),
    method<moe_combine, 4, 2>("moe_combine"),
    method<moe_combine_backward, 6, 4, 5>("moe_combine_backward"),
    method<gemm_w4, 12, 2>("gemm_w4"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_ops(void) { return PyModule_Create(&module); }
