// The host side of the Python calls in ops.py: checks tensors, allocates
// outputs and calls the C ABI. These operators run for a few microseconds at
// the sizes of a decoding loop, where the same checks in Python cost more
// than the launch (norm of one token 11 us, a step of 36 tensors 47 us; here
// 6 and 7).
//
// A CPython module without state but the addresses of the C ABI's functions,
// which ops.py hands over once (bind): the library stays loaded by _lib.py
// alone. Every function takes the stream as an integer and returns its
// tensors, or the status of a call that the library refused; what does not
// fit is a ValueError, raised before anything is enqueued.
#include <torch/csrc/python_headers.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <stdexcept>
#include <string>
#include <utility>
#include <vector>

#include "mok.h"

namespace {

decltype(&mok_rms_norm) f_rms_norm;
decltype(&mok_rms_norm_scratch_bytes) f_rms_norm_scratch_bytes;
decltype(&mok_rms_norm_backward) f_rms_norm_backward;
decltype(&mok_router_scratch_bytes) f_router_scratch_bytes;
decltype(&mok_router_topk) f_router_topk;
decltype(&mok_router_topk_backward) f_router_topk_backward;
decltype(&mok_adamw_step) f_adamw_step;
decltype(&mok_grouped_matmul_scratch_bytes) f_grouped_matmul_scratch_bytes;
decltype(&mok_grouped_matmul) f_grouped_matmul;
decltype(&mok_grouped_matmul_dx) f_grouped_matmul_dx;
decltype(&mok_grouped_matmul_dw) f_grouped_matmul_dw;
decltype(&mok_w4_quantize) f_w4_quantize;
decltype(&mok_w4_dequantize) f_w4_dequantize;
decltype(&mok_w4_matmul) f_w4_matmul;
decltype(&mok_forward_w4_scratch_bytes) f_forward_w4_scratch_bytes;
decltype(&mok_forward_w4) f_forward_w4;

using at::Tensor;
constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kU8 = at::kByte;

[[noreturn]] void bad(const std::string& what) { throw std::invalid_argument(what); }

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}
const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    case at::kDouble: return "torch.float64";
    case at::kByte: return "torch.uint8";
    case at::kBool: return "torch.bool";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    case at::kFloat8_e8m0fnu: return "torch.float8_e8m0fnu";
    default: return "another type";
  }
}
using Types = std::initializer_list<at::ScalarType>;
std::string text(Types ts) {
  std::string r;
  for (auto t : ts) r += (r.empty() ? "" : " or ") + std::string(name_of(t));
  return r;
}
bool one_of(at::ScalarType t, Types ts) { return std::find(ts.begin(), ts.end(), t) != ts.end(); }

const Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
// A tensor or None (null).
const Tensor* maybe(const char* name, PyObject* o) { return o == Py_None ? nullptr : &tensor(name, o); }

const Tensor& on_gpu(const char* name, const Tensor& t) {
  if (!t.is_cuda()) bad(std::string(name) + " must live on the GPU (a CUDA tensor)");
  return t;
}
void check(const char* name, const Tensor& t, const Tensor& ref, Types types) {
  if (t.device() != ref.device())
    bad(std::string(name) + " is on " + t.device().str() + ", not on " + ref.device().str());
  if (!one_of(t.scalar_type(), types))
    bad(std::string(name) + " must be " + text(types) + ", got " + name_of(t.scalar_type()));
}
void shaped(const char* name, const Tensor& t, at::IntArrayRef want) {
  if (t.sizes() != want) bad(std::string(name) + " must have shape " + text(want) + ", got " + text(t.sizes()));
}
void* dense(const char* name, const Tensor& t) {
  if (!t.is_contiguous()) bad(std::string(name) + " must be contiguous");
  return t.data_ptr();
}
// Row stride of a tensor whose last dimension is dense and whose rows lie at one stride.
int64_t row_stride(const char* name, const Tensor& t) {
  if (t.is_contiguous()) return t.size(-1);
  if (t.dim() != 2 || (t.stride(1) != 1 && t.size(1) > 1) || t.stride(0) < t.size(1))
    bad(std::string(name) + " must be contiguous, or 2-D with dense rows that do not overlap");
  return t.stride(0);
}
void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
Tensor make(at::IntArrayRef sizes, const Tensor& like, at::ScalarType type) {
  return at::empty(sizes, like.options().dtype(type).requires_grad(false));
}
bool fp32(const Tensor& t) { return t.scalar_type() == kF32; }

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int32_t small_integer(const char* name, PyObject* o) {
  const int64_t v = integer(o);
  if (v != (int32_t)v) bad(std::string(name) + " is out of range");
  return (int32_t)v;
}
void* stream_of(PyObject* o) {
  void* s = PyLong_AsVoidPtr(o);
  if (!s && PyErr_Occurred()) throw python_error();
  return s;
}
void count(const char* name, Py_ssize_t have, Py_ssize_t want) {
  if (have != want) bad(std::string(name) + " takes " + std::to_string(want) + " arguments");
}

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
// A tuple of tensors (undefined ones None), or the status of a refused call.
PyObject* result(mok_status st, std::initializer_list<Tensor> ts) {
  if (st != MOK_OK) return PyLong_FromLong(st);
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
  return r;
}

// Moves the in-place version counter of a tensor that a call wrote through its
// address: autograd's check of saved tensors and the layer's quantized weights
// go by it. (Tensors made in inference mode have none.)
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(const Tensor* t) {
  if (t) written(*t);
}
// Whether a call may have enqueued work: not if its arguments were refused.
bool ran(mok_status st) { return st == MOK_OK || st == MOK_ERR_HIP; }

// The memory between a tensor's first and last element.
std::pair<uintptr_t, uintptr_t> span(const Tensor& t) {
  const uintptr_t p = (uintptr_t)t.data_ptr();
  int64_t last = 0;
  for (int64_t i = 0; i < t.dim(); ++i) last += (t.size(i) - 1) * t.stride(i);
  return {p, t.numel() ? p + (last + 1) * t.element_size() : p};
}
// Refuses a given output that overlaps `other` (null: none): another row's
// threads would read what one has written. `in_place`: where `other` is the
// same memory, element by element, a row is read before it is written.
void apart(const char* name, const Tensor& out, const char* other_name, const Tensor* other, bool in_place) {
  if (!other) return;
  const auto a = span(out), b = span(*other);
  if (a.first >= b.second || b.first >= a.second) return;
  if (in_place && a == b && out.element_size() == other->element_size() && other->is_contiguous()) return;
  bad(std::string(name) + " overlaps " + other_name);
}

// ---- RMS norm ----

struct Norm {
  const Tensor &x, &w;
  const Tensor* res;
  int64_t cols, ldx, ldr = 0;
  Tensor sum;
  Norm(PyObject* const* a) : x(on_gpu("x", tensor("x", a[0]))), w(tensor("weight", a[1])), res(maybe("residual", a[2])) {
    cols = x.dim() ? x.size(-1) : 0;
    if (cols < 1) bad("x must have a last dimension of at least 1");
    check("x", x, x, {kBf16, kF32});
    check("weight", w, x, {kBf16, kF32});
    shaped("weight", w, {cols});
    dense("weight", w);
    ldx = row_stride("x", x);
    if (res) {
      check("residual", *res, x, {kBf16, kF32});
      shaped("residual", *res, x.sizes());
      ldr = row_stride("residual", *res);
    }
  }
  mok_status run(double eps, void* y, void* codes, void* scale, void* rstd, void* stream) {
    if (res) sum = make(x.sizes(), x, res->scalar_type());
    return f_rms_norm(x.data_ptr(), fp32(x), ldx, ptr(res), res && fp32(*res), ldr, w.data_ptr(), fp32(w),
                      x.numel() / cols, cols, (float)eps, sum.defined() ? sum.data_ptr() : nullptr, y, (uint8_t*)codes,
                      (uint8_t*)scale, (float*)rstd, stream);
  }
};

// rms_norm(x, weight, residual, eps, stream) -> (y, sum, rstd)
PyObject* rms_norm(PyObject* const* a, Py_ssize_t n) {
  count("rms_norm", n, 5);
  Norm k(a);
  Tensor y = make(k.x.sizes(), k.x, kBf16), rstd = make(k.x.sizes().slice(0, k.x.dim() - 1), k.x, kF32);
  const mok_status st = k.run(number(a[3]), y.data_ptr(), nullptr, nullptr, rstd.data_ptr(), stream_of(a[4]));
  return result(st, {y, k.sum, rstd});
}

// rms_norm_mxfp8(x, weight, residual, eps, y, rstd, stream) -> (codes, scale, sum)
PyObject* rms_norm_mxfp8(PyObject* const* a, Py_ssize_t n) {
  count("rms_norm_mxfp8", n, 7);
  Norm k(a);
  if (k.cols % 32 != 0) bad("MXFP8 needs a last dimension that is a multiple of 32");
  const auto lead = k.x.sizes().slice(0, k.x.dim() - 1);
  const Tensor *y = maybe("y", a[4]), *rstd = maybe("rstd", a[5]);
  if (y) check("y", *y, k.x, {kBf16}), shaped("y", *y, k.x.sizes()), dense("y", *y);
  if (rstd) check("rstd", *rstd, k.x, {kF32}), shaped("rstd", *rstd, lead), dense("rstd", *rstd);
  if (y) apart("y", *y, "x", &k.x, true), apart("y", *y, "residual", k.res, true), apart("y", *y, "weight", &k.w, false);
  if (rstd) {
    apart("rstd", *rstd, "x", &k.x, false), apart("rstd", *rstd, "residual", k.res, false);
    apart("rstd", *rstd, "weight", &k.w, false), apart("rstd", *rstd, "y", y, false);
  }
  auto blocks = lead.vec();
  blocks.push_back(k.cols / 32);
  Tensor codes = make(k.x.sizes(), k.x, kU8), scale = make(blocks, k.x, kU8);
  const mok_status st = k.run(number(a[3]), ptr(y), codes.data_ptr(), scale.data_ptr(), ptr(rstd), stream_of(a[6]));
  if (ran(st)) written(y), written(rstd);
  return result(st, {codes, scale, k.sum});
}

// rms_norm_backward(dy, s, rstd, weight, d_sum, dx, stream) -> (ds, d_weight)
PyObject* rms_norm_backward(PyObject* const* a, Py_ssize_t n) {
  count("rms_norm_backward", n, 7);
  const Tensor &dy = on_gpu("dy", tensor("dy", a[0])), &s = tensor("s", a[1]), &rstd = tensor("rstd", a[2]),
               &w = tensor("weight", a[3]);
  const Tensor *dsum = maybe("d_sum", a[4]), *dx = maybe("dx", a[5]);
  const int64_t cols = dy.dim() ? dy.size(-1) : 0;
  if (cols < 1) bad("dy must have a last dimension of at least 1");
  check("dy", dy, dy, {kBf16});
  check("s", s, dy, {kBf16, kF32});
  shaped("s", s, dy.sizes());
  check("rstd", rstd, dy, {kF32});
  shaped("rstd", rstd, dy.sizes().slice(0, dy.dim() - 1));
  check("weight", w, dy, {kBf16, kF32});
  shaped("weight", w, {cols});
  const int64_t lddy = row_stride("dy", dy), lds = row_stride("s", s);
  int64_t ldd = 0;
  if (dsum) {
    check("d_sum", *dsum, dy, {s.scalar_type()});
    shaped("d_sum", *dsum, dy.sizes());
    ldd = row_stride("d_sum", *dsum);
  }
  if (dx) check("dx", *dx, dy, {kBf16}), shaped("dx", *dx, dy.sizes()), dense("dx", *dx);
  if (dx) {
    apart("dx", *dx, "dy", &dy, true), apart("dx", *dx, "s", &s, true), apart("dx", *dx, "d_sum", dsum, true);
    apart("dx", *dx, "rstd", &rstd, false), apart("dx", *dx, "weight", &w, false);
  }
  const void* pr = dense("rstd", rstd);
  const void* pw = dense("weight", w);
  const int64_t rows = dy.numel() / cols;
  Tensor ds = make(s.sizes(), s, s.scalar_type()), dw = make({cols}, w, w.scalar_type());
  const size_t bytes = f_rms_norm_scratch_bytes(rows, cols);
  Tensor scratch = make({(int64_t)bytes}, dy, kU8);
  const mok_status st = f_rms_norm_backward(dy.data_ptr(), lddy, s.data_ptr(), fp32(s), lds, (const float*)pr, pw,
                                            fp32(w), ptr(dsum), ldd, rows, cols, ds.data_ptr(), ptr(dx), dw.data_ptr(),
                                            scratch.data_ptr(), bytes, stream_of(a[6]));
  if (ran(st)) written(dx);
  return result(st, {ds, dw});
}

// ---- router ----

struct Router {
  const Tensor& l;
  const Tensor *bias, *mask;
  int64_t T, E, ld;
  Router(PyObject* logits, PyObject* b, PyObject* m)
      : l(on_gpu("logits", tensor("logits", logits))), bias(maybe("bias", b)), mask(maybe("token_mask", m)) {
    if (l.dim() != 2) bad("logits must be [tokens, experts]");
    check("logits", l, l, {kBf16, kF32});
    T = l.size(0), E = l.size(1);
    if (E < 1 || E > 1 << 20) bad("logits must have between 1 and 2^20 experts");
    ld = row_stride("logits", l);
    if (bias) check("bias", *bias, l, {kF32}), shaped("bias", *bias, {E}), dense("bias", *bias);
    if (mask) check("token_mask", *mask, l, {at::kBool, kU8}), shaped("token_mask", *mask, {T}), dense("token_mask", *mask);
  }
};

// router_topk(logits, k, scoring, renormalize, scale, bias, token_mask, losses, stream)
//   -> (weights, ids, counts, losses)
PyObject* router_topk(PyObject* const* a, Py_ssize_t n) {
  count("router_topk", n, 9);
  const Router r(a[0], a[5], a[6]);
  const int32_t k = small_integer("k", a[1]);
  if (k < 1) bad("k must be at least 1");
  const bool stats = a[7] == Py_True;
  Tensor weights = make({r.T, k}, r.l, kF32), ids = make({r.T, k}, r.l, at::kLong), counts, losses, scratch;
  size_t bytes = 0;
  if (stats) {
    counts = make({r.E + 1}, r.l, at::kInt);
    losses = make({2}, r.l, kF32);
    bytes = f_router_scratch_bytes(r.T, (int32_t)r.E);
    scratch = make({(int64_t)bytes}, r.l, kU8);
  }
  const mok_status st = f_router_topk(
      r.l.data_ptr(), fp32(r.l), r.T, r.ld, (int32_t)r.E, k, (const float*)ptr(r.bias), (const uint8_t*)ptr(r.mask),
      small_integer("scoring", a[2]), a[3] == Py_True, (float)number(a[4]), weights.data_ptr<float>(),
      ids.data_ptr<int64_t>(), stats ? counts.data_ptr<int32_t>() : nullptr, stats ? losses.data_ptr<float>() : nullptr,
      stats ? scratch.data_ptr() : nullptr, bytes, stream_of(a[8]));
  return result(st, {weights, ids, counts, losses});
}

// router_topk_backward(d_weights, logits, ids, scoring, renormalize, scale, bias, token_mask, counts, d_losses, stream)
//   -> (d_logits,)
PyObject* router_topk_backward(PyObject* const* a, Py_ssize_t n) {
  count("router_topk_backward", n, 11);
  const Router r(a[1], a[6], a[7]);
  const Tensor &dw = tensor("d_weights", a[0]), &ids = tensor("ids", a[2]);
  const Tensor *counts = maybe("counts", a[8]), *dl = maybe("d_losses", a[9]);
  if (ids.dim() != 2) bad("ids must be [tokens, k]");
  const int64_t k = ids.size(1);
  if (k < 1 || k > 1 << 20) bad("ids must have between 1 and 2^20 columns");
  check("ids", ids, r.l, {at::kLong});
  shaped("ids", ids, {r.T, k});
  check("d_weights", dw, r.l, {kF32});
  shaped("d_weights", dw, {r.T, k});
  if ((counts == nullptr) != (dl == nullptr)) bad("counts and d_losses come together");
  if (counts) {
    check("counts", *counts, r.l, {at::kInt}), shaped("counts", *counts, {r.E + 1}), dense("counts", *counts);
    check("d_losses", *dl, r.l, {kF32}), shaped("d_losses", *dl, {2}), dense("d_losses", *dl);
  }
  const void* pdw = dense("d_weights", dw);
  const void* pids = dense("ids", ids);
  Tensor d = make({r.T, r.E}, r.l, r.l.scalar_type());
  const mok_status st = f_router_topk_backward(
      (const float*)pdw, r.l.data_ptr(), fp32(r.l), r.T, r.ld, (int32_t)r.E, (int32_t)k, (const float*)ptr(r.bias),
      (const uint8_t*)ptr(r.mask), small_integer("scoring", a[3]), a[4] == Py_True, (float)number(a[5]),
      (const int64_t*)pids, (const int32_t*)ptr(counts), (const float*)ptr(dl), d.data_ptr(), stream_of(a[10]));
  return result(st, {d});
}

// ---- AdamW ----

// A list or tuple, held while its items are in use.
struct Items {
  PyObject* fast;
  Items(const char* name, PyObject* o) : fast(nullptr) {
    if (!PyList_Check(o) && !PyTuple_Check(o)) bad(std::string(name) + " must be a list or tuple");
    fast = o;
    Py_INCREF(fast);
  }
  Items(const Items&) = delete;
  ~Items() { Py_DECREF(fast); }
  int size() const { return (int)PySequence_Fast_GET_SIZE(fast); }
  PyObject* operator[](int i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

struct Step {
  int n = 0;
  std::vector<int64_t> numels;
  struct Bytes {
    uintptr_t begin, end;
    bool written;
  };
  std::vector<Bytes> touched;  // what the step reads and writes, tensor by tensor, one of each list
  size_t lists = 0;
  Bytes scale{0, 0, false};
  std::vector<const Tensor*> outputs;
  const Tensor* first = nullptr;

  // Adds one tensor of a list: all of one type of `types`, dense, on one GPU.
  void add(const char* name, const Tensor& t, Types types, int64_t numel, at::ScalarType* type,
           std::vector<void*>* to, bool writes) {
    if (t.device() != first->device()) bad("every tensor must be on " + first->device().str() + ": " + name);
    if (t.numel() != numel) bad(std::string("the tensors of ") + name + " must have the sizes of the params");
    if (to->empty() && one_of(t.scalar_type(), types)) *type = t.scalar_type();
    if (t.scalar_type() != *type)
      bad(std::string(name) + " must all be " + text(types) + ", got " + name_of(t.scalar_type()));
    if (!t.is_contiguous()) bad(std::string("every tensor of ") + name + " must be contiguous");
    void* p = t.data_ptr();
    to->push_back(p);
    if (writes) outputs.push_back(&t);
    if (numel > 0) touched.push_back({(uintptr_t)p, (uintptr_t)p + numel * t.element_size(), writes});
  }
  // Whether a range that is written overlaps another. A list's tensors mostly
  // lie in memory in their order: the lists are a few ascending runs, which are
  // merged (36 tensors, 4 lists: 0.4 us; a sort takes 1.5).
  bool overlaps() const {
    const auto before = [](const Bytes& x, const Bytes& y) { return x.begin < y.begin; };
    constexpr size_t kRuns = 16;
    size_t run[kRuns + 1], runs = 0;  // where each begins, and the end
    const size_t n = touched.size() + (scale.end ? 1 : 0);
    std::vector<Bytes> both(2 * n);
    Bytes *a = both.data(), *b = a + n, *to = a;
    const auto next = [&](const Bytes& x) {
      if (to == a || before(x, to[-1])) {
        if (runs < kRuns) run[runs] = to - a;
        ++runs;
      }
      *to++ = x;
    };
    for (size_t l = 0; l < lists; ++l)
      for (size_t i = l; i < touched.size(); i += lists) next(touched[i]);
    if (scale.end) next(scale);
    if (runs > kRuns) {
      std::sort(a, a + n, before);
    } else {
      run[runs] = n;
      for (size_t left = runs; left > 1; left = (left + 1) / 2, std::swap(a, b)) {
        for (size_t i = 0; i < left; i += 2) {
          const size_t mid = run[i + 1], end = i + 1 < left ? run[i + 2] : mid;
          std::merge(a + run[i], a + mid, a + mid, a + end, b + run[i], before);
          run[i / 2] = run[i];
        }
        run[(left + 1) / 2] = n;
      }
    }
    uintptr_t any_end = 0, written_end = 0;
    for (size_t i = 0; i < n; ++i) {
      const Bytes& x = a[i];
      if (x.begin < (x.written ? any_end : written_end)) return true;
      any_end = std::max(any_end, x.end);
      if (x.written) written_end = std::max(written_end, x.end);
    }
    return false;
  }
  void length(const char* name, const Items& l) const {
    if (l.size() != n)
      bad(std::string(name) + " has " + std::to_string(l.size()) + " tensors, params " + std::to_string(n));
  }
};

// adamw_step(params, grads, exp_avgs, exp_avg_sqs, masters, step, lr, beta1, beta2, eps, weight_decay, grad_scale,
//            seed, stream) -> status
PyObject* adamw_step(PyObject* const* a, Py_ssize_t nargs) {
  count("adamw_step", nargs, 14);
  const Items params("params", a[0]), grads("grads", a[1]), ms("exp_avgs", a[2]), vs("exp_avg_sqs", a[3]);
  const bool with_masters = a[4] != Py_None;
  const Items masters("masters", with_masters ? a[4] : a[0]);
  Step s;
  s.n = params.size();
  s.length("grads", grads), s.length("exp_avgs", ms), s.length("exp_avg_sqs", vs), s.length("masters", masters);
  if (s.n == 0) return PyLong_FromLong(MOK_OK);
  s.first = &on_gpu("params", tensor("params", params[0]));
  const bool small = !THPVariable_Check(ms[0]);
  constexpr auto kNone = at::ScalarType::Undefined;
  at::ScalarType pt = kNone, gt = kNone, wt = kNone, mt[2] = {kNone, kNone}, st[2] = {kNone, kNone};
  std::vector<void*> pp, pg, pw, pm[2], psc[2];
  for (auto* v : {&pp, &pg, &pw, &pm[0], &pm[1], &psc[0], &psc[1]}) v->reserve(s.n);
  s.numels.reserve(s.n);
  s.touched.reserve((size_t)s.n * 7);
  s.lists = (small ? 6 : 4) + (with_masters ? 1 : 0);
  s.outputs.reserve((size_t)s.n * 6);
  for (int i = 0; i < s.n; ++i) {
    const Tensor& p = tensor("params", params[i]);
    const int64_t n = p.numel();
    s.numels.push_back(n);
    s.add("params", p, {kBf16, kF32}, n, &pt, &pp, true);
    s.add("grads", tensor("grads", grads[i]), {kBf16, kF32}, n, &gt, &pg, false);
    if (with_masters) {
      if (pt != kBf16) bad("masters go with bf16 params");
      s.add("masters", tensor("masters", masters[i]), {kF32}, n, &wt, &pw, true);
    }
    for (int k = 0; k < 2; ++k) {
      const char* name = k ? "exp_avg_sqs" : "exp_avgs";
      PyObject* o = k ? vs[i] : ms[i];
      if (!small) {
        s.add(name, tensor(name, o), {kF32}, n, &mt[k], &pm[k], true);
        continue;
      }
      if (!(PyTuple_Check(o) || PyList_Check(o)) || PySequence_Fast_GET_SIZE(o) != 2)
        bad(std::string(name) + " must be pairs (codes, scale)");
      s.add(name, tensor(name, PySequence_Fast_GET_ITEM(o, 0)), {kU8, at::kFloat8_e4m3fn}, n, &mt[k], &pm[k], true);
      s.add(k ? "exp_avg_sqs scales" : "exp_avgs scales", tensor(name, PySequence_Fast_GET_ITEM(o, 1)), {kU8, at::kFloat8_e8m0fnu},
            (n + 31) / 32, &st[k], &psc[k], true);
    }
  }
  const Tensor* scale = maybe("grad_scale", a[11]);
  if (scale) {
    check("grad_scale", *scale, *s.first, {kF32});
    if (scale->numel() != 1) bad("grad_scale must have one element");
    s.scale = {(uintptr_t)scale->data_ptr(), (uintptr_t)scale->data_ptr() + sizeof(float), false};
  }
  if (s.overlaps()) bad("a tensor that the step writes is given twice, or overlaps another");
  mok_adamw u{};
  u.struct_size = sizeof(u);
  u.count = s.n;
  u.params = pp.data();
  u.grads = (const void* const*)pg.data();
  u.masters = with_masters ? pw.data() : nullptr;
  u.exp_avgs = pm[0].data(), u.exp_avg_sqs = pm[1].data();
  u.exp_avg_scales = small ? psc[0].data() : nullptr, u.exp_avg_sq_scales = small ? psc[1].data() : nullptr;
  u.numels = s.numels.data();
  u.grad_scale = (const float*)ptr(scale);
  u.step = integer(a[5]);
  u.lr = number(a[6]), u.beta1 = number(a[7]), u.beta2 = number(a[8]), u.eps = number(a[9]);
  u.weight_decay = number(a[10]);
  u.param_fp32 = pt == kF32, u.grad_fp32 = gt == kF32, u.state_bits = small ? 8 : 32;
  u.seed = (uint32_t)PyLong_AsUnsignedLongMask(a[12]);
  if (PyErr_Occurred()) throw python_error();
  const mok_status status = f_adamw_step(&u, stream_of(a[13]));
  if (ran(status))
    for (const Tensor* t : s.outputs) written(*t);
  return PyLong_FromLong(status);
}

// ---- grouped products ----

// The weight [experts, n, k], the offsets [experts + 1] and rows [rows, cols] of a grouped product.
struct Grouped {
  const Tensor &w, &offsets;
  int64_t E, n, k;
  Grouped(PyObject* weight, PyObject* off, const Tensor& first) : w(tensor("weight", weight)), offsets(tensor("offsets", off)) {
    check("weight", w, first, {kBf16});
    if (w.dim() != 3 || w.size(0) < 1 || w.size(1) < 1 || w.size(2) < 1) bad("weight must be [experts, n, k], none of them 0");
    dense("weight", w);
    E = w.size(0), n = w.size(1), k = w.size(2);
    if (E > 1024) bad("at most 1024 experts");
    check("offsets", offsets, first, {at::kInt, at::kLong});
    shaped("offsets", offsets, {E + 1});
    dense("offsets", offsets);
  }
  int wide() const { return offsets.scalar_type() == at::kLong; }
  // The scratch that a product of `rows` rows can use (undefined: none).
  Tensor scratch(mok_grouped_op op, int64_t rows) const {
    const size_t bytes = f_grouped_matmul_scratch_bytes(op, rows, (int32_t)E, n, k);
    return bytes ? make({(int64_t)bytes}, w, kU8) : Tensor();
  }
};
void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
size_t bytes_of(const Tensor& t) { return t.defined() ? t.nbytes() : 0; }
int64_t rows_of(const char* name, const Tensor& t, const Tensor& first, int64_t cols) {
  check(name, t, first, {kBf16});
  if (t.dim() != 2 || t.size(1) != cols) bad(std::string(name) + " must be [rows, " + std::to_string(cols) + "], got " + text(t.sizes()));
  return t.size(0);
}

// grouped_matmul(x, weight, offsets, out, stream) -> (y,)
PyObject* grouped_matmul(PyObject* const* a, Py_ssize_t nargs) {
  count("grouped_matmul", nargs, 5);
  const Tensor& x = on_gpu("x", tensor("x", a[0]));
  const Grouped g(a[1], a[2], x);
  const int64_t rows = rows_of("x", x, x, g.k), ldx = row_stride("x", x);
  const Tensor* out = maybe("out", a[3]);
  if (out) {
    if (rows_of("out", *out, x, g.n) != rows) bad("out must have x's rows");
    apart("out", *out, "x", &x, false), apart("out", *out, "weight", &g.w, false);
    apart("out", *out, "offsets", &g.offsets, false);
  }
  Tensor y = out ? *out : make({rows, g.n}, x, kBf16);
  const int64_t ldy = row_stride("out", y);
  const Tensor scratch = g.scratch(MOK_GROUPED_Y, rows);
  const mok_status st = f_grouped_matmul(x.data_ptr(), ldx, g.w.data_ptr(), g.offsets.data_ptr(), g.wide(), rows,
                                         (int32_t)g.E, g.n, g.k, y.data_ptr(), ldy, !out, ptr(scratch),
                                         bytes_of(scratch), stream_of(a[4]));
  if (ran(st)) written(out);
  return result(st, {y});
}

// grouped_matmul_backward(dy, x, weight, offsets, need_dx, need_dw, dw_fp32, stream) -> (dx, dw)
PyObject* grouped_matmul_backward(PyObject* const* a, Py_ssize_t nargs) {
  count("grouped_matmul_backward", nargs, 8);
  const Tensor &dy = on_gpu("dy", tensor("dy", a[0])), &x = tensor("x", a[1]);
  const Grouped g(a[2], a[3], dy);
  const int64_t rows = rows_of("dy", dy, dy, g.n), lddy = row_stride("dy", dy);
  if (rows_of("x", x, dy, g.k) != rows) bad("x must have dy's rows");
  const int64_t ldx = row_stride("x", x);
  const bool wide = a[6] == Py_True;
  Tensor dx, dw;
  mok_status st = MOK_OK;
  if (a[4] == Py_True) {
    dx = make({rows, g.k}, dy, kBf16);
    const Tensor scratch = g.scratch(MOK_GROUPED_DX, rows);
    st = f_grouped_matmul_dx(dy.data_ptr(), lddy, g.w.data_ptr(), g.offsets.data_ptr(), g.wide(), rows, (int32_t)g.E,
                             g.n, g.k, dx.data_ptr(), g.k, 1, ptr(scratch), bytes_of(scratch), stream_of(a[7]));
  }
  if (st == MOK_OK && a[5] == Py_True) {
    dw = make({g.E, g.n, g.k}, dy, wide ? kF32 : kBf16);
    const Tensor scratch = g.scratch(MOK_GROUPED_DW, rows);
    st = f_grouped_matmul_dw(dy.data_ptr(), lddy, x.data_ptr(), ldx, g.offsets.data_ptr(), g.wide(), rows, (int32_t)g.E,
                             g.n, g.k, dw.data_ptr(), wide, ptr(scratch), bytes_of(scratch), stream_of(a[7]));
  }
  return result(st, {dx, dw});
}

// ---- 4-bit weights ----

struct Weight4 {
  const Tensor &codes, &scale;
  const Tensor* zero;
  int32_t format, group = 0;
  int64_t k = 0;
  // Checks types, devices and that the three fit each other. `name`: the weight's.
  Weight4(const char* name, PyObject* c, PyObject* s, PyObject* z, const Tensor& first)
      : codes(tensor(name, c)), scale(tensor((std::string(name) + "'s scale").c_str(), s)), zero(maybe("a zero point", z)) {
    const std::string n(name);
    check(name, codes, first, {kU8});
    check((n + "'s scale").c_str(), scale, first, {kBf16, kU8, at::kFloat8_e8m0fnu});
    format = scale.scalar_type() == kBf16 ? MOK_W4_INT4 : MOK_W4_MXFP4;
    if (codes.dim() < 1 || codes.size(-1) < 1) bad(n + " must have a last dimension of at least 1");
    k = codes.size(-1) * 2;
    if (scale.dim() != codes.dim() || scale.sizes().slice(0, codes.dim() - 1) != codes.sizes().slice(0, codes.dim() - 1))
      bad(n + "'s scale must have its rows: codes " + text(codes.sizes()) + ", scale " + text(scale.sizes()));
    const int64_t groups = scale.size(-1);
    if (groups < 1 || k % groups != 0 || (k / groups != 32 && (format == MOK_W4_MXFP4 || (k / groups != 64 && k / groups != 128))))
      bad(n + ": " + std::to_string(groups) + " scales for " + std::to_string(k) + " columns are no groups of 32" +
          (format == MOK_W4_MXFP4 ? "" : ", 64 or 128"));
    group = (int32_t)(k / groups);
    dense(name, codes), dense((n + "'s scale").c_str(), scale);
    if (zero) {
      if (format == MOK_W4_MXFP4) bad("MXFP4 weights have no zero points");
      check((n + "'s zero point").c_str(), *zero, first, {kU8});
      shaped((n + "'s zero point").c_str(), *zero, scale.sizes());
      dense((n + "'s zero point").c_str(), *zero);
    }
  }
  mok_w4 c() const { return mok_w4{(const uint8_t*)codes.data_ptr(), scale.data_ptr(), (const uint8_t*)ptr(zero)}; }
  int64_t rows() const { return codes.numel() / codes.size(-1); }
};

// w4_quantize(weight, mxfp4, group, zero_point, stream) -> (codes, scale, zero)
PyObject* w4_quantize(PyObject* const* a, Py_ssize_t nargs) {
  count("w4_quantize", nargs, 5);
  const Tensor& w = on_gpu("weight", tensor("weight", a[0]));
  check("weight", w, w, {kBf16, kF32});
  const bool mx = a[1] == Py_True, with_zero = a[3] == Py_True;
  const int32_t group = small_integer("group", a[2]);
  if (mx && (with_zero || group != 32)) bad("MXFP4 has groups of 32 and no zero points");
  if (group != 32 && group != 64 && group != 128) bad("group must be 32, 64 or 128");
  if (w.dim() < 1 || w.size(-1) < 1 || w.size(-1) % group != 0) bad("the last dimension must be a multiple of the group, " + std::to_string(group));
  const int64_t cols = w.size(-1), ld = row_stride("weight", w);
  auto size = w.sizes().vec();
  size.back() = cols / 2;
  Tensor codes = make(size, w, kU8), zero;
  size.back() = cols / group;
  Tensor scale = make(size, w, mx ? kU8 : kBf16);
  if (with_zero) zero = make(size, w, kU8);
  const mok_status st = f_w4_quantize(w.data_ptr(), fp32(w), w.numel() / cols, cols, ld, mx ? MOK_W4_MXFP4 : MOK_W4_INT4,
                                      group, (uint8_t*)codes.data_ptr(), scale.data_ptr(),
                                      with_zero ? (uint8_t*)zero.data_ptr() : nullptr, stream_of(a[4]));
  return result(st, {codes, scale, zero});
}

// w4_dequantize(codes, scale, zero, stream) -> (values,)
PyObject* w4_dequantize(PyObject* const* a, Py_ssize_t nargs) {
  count("w4_dequantize", nargs, 4);
  const Weight4 w("codes", a[0], a[1], a[2], on_gpu("codes", tensor("codes", a[0])));
  auto size = w.codes.sizes().vec();
  size.back() = w.k;
  Tensor out = make(size, w.codes, kBf16);
  const mok_w4 c = w.c();
  const mok_status st = f_w4_dequantize(&c, w.rows(), w.k, w.format, w.group, out.data_ptr(), stream_of(a[3]));
  return result(st, {out});
}

// w4_matmul(x, codes, scale, zero, stream) -> (y,)
PyObject* w4_matmul(PyObject* const* a, Py_ssize_t nargs) {
  count("w4_matmul", nargs, 5);
  const Tensor& x = on_gpu("x", tensor("x", a[0]));
  check("x", x, x, {kBf16});
  const Weight4 w("codes", a[1], a[2], a[3], x);
  if (w.codes.dim() != 2 || w.codes.size(0) < 1) bad("codes must be [n, k/2]");
  if (x.dim() < 1 || x.size(-1) != w.k) bad("x must have a last dimension of " + std::to_string(w.k));
  const int64_t n = w.codes.size(0), T = x.numel() / w.k, ldx = row_stride("x", x);
  auto size = x.sizes().vec();
  size.back() = n;
  Tensor y = make(size, x, kBf16);
  const mok_w4 c = w.c();
  const mok_status st = f_w4_matmul(x.data_ptr(), ldx, T, n, w.k, w.format, w.group, &c, y.data_ptr(), n, stream_of(a[4]));
  return result(st, {y});
}

// forward_w4(x, router_weights, top_experts, weights, limit, out, stream) -> (y,); weights: codes, scale and zero (or
// None) of routed gate, up, down and of shared gate, up, down (or None)
PyObject* forward_w4(PyObject* const* a, Py_ssize_t nargs) {
  count("forward_w4", nargs, 7);
  const Tensor &x = on_gpu("x", tensor("x", a[0])), &rw = tensor("router_weights", a[1]), &ids = tensor("top_experts", a[2]);
  check("x", x, x, {kBf16});
  if (x.dim() != 2 || x.size(1) < 1) bad("x must be [tokens, hidden]");
  const int64_t T = x.size(0), H = x.size(1);
  check("router_weights", rw, x, {kF32});
  check("top_experts", ids, x, {at::kLong});
  if (ids.dim() != 2 || ids.size(0) != T || ids.size(1) < 1 || ids.size(1) > 64)
    bad("top_experts must be [tokens, topk], topk between 1 and 64, got " + text(ids.sizes()));
  shaped("router_weights", rw, ids.sizes());
  if (!PyTuple_Check(a[3]) || PyTuple_GET_SIZE(a[3]) != 18) bad("weights must be 18 entries");
  static const char* const names[6] = {"routed_gate", "routed_up", "routed_down", "shared_gate", "shared_up", "shared_down"};
  mok_w4_layer l{};
  l.struct_size = sizeof(l);
  mok_w4* to[6] = {&l.routed_gate, &l.routed_up, &l.routed_down, &l.shared_gate, &l.shared_up, &l.shared_down};
  int64_t E = 0, I = 0, Is = 0;
  bool with_zero = false;
  const Tensor* out = maybe("out", a[5]);
  for (int i = 0; i < 6; ++i) {
    PyObject* const* part = &PyTuple_GET_ITEM(a[3], 3 * i);
    if (i >= 3 && part[0] == Py_None) {
      if (i > 3 && Is) bad("the shared expert needs all of shared_gate, shared_up and shared_down");
      if (part[1] != Py_None || part[2] != Py_None) bad(std::string(names[i]) + "'s codes are missing");
      continue;
    }
    if (i > 3 && !Is) bad("the shared expert needs all of shared_gate, shared_up and shared_down");
    const Weight4 w(names[i], part[0], part[1], part[2], x);
    if (i == 0) {
      if (w.codes.dim() != 3 || w.codes.size(0) < 1 || w.codes.size(0) > 1024 || w.codes.size(1) < 1)
        bad("routed_gate must be [experts, intermediate, hidden/2], at most 1024 experts");
      E = w.codes.size(0), I = w.codes.size(1);
      l.format = w.format, l.group = w.group, with_zero = w.zero != nullptr;
    }
    if (i == 3) {
      if (w.codes.dim() != 2 || w.codes.size(0) < 1) bad("shared_gate must be [shared_intermediate, hidden/2]");
      Is = w.codes.size(0);
    }
    const int64_t wide = i < 3 ? I : Is, n = i % 3 == 2 ? H : wide, k = i % 3 == 2 ? wide : H;
    if (k % 2 != 0) bad("hidden and intermediate must be even");
    if (i < 3)
      shaped(names[i], w.codes, {E, n, k / 2});
    else
      shaped(names[i], w.codes, {n, k / 2});
    if (w.format != l.format || w.group != l.group || (w.zero != nullptr) != with_zero)
      bad("all weights must have one format and group, and zero points in all of them or in none");
    *to[i] = w.c();
    if (out) apart("out", *out, names[i], &w.codes, false), apart("out", *out, names[i], &w.scale, false), apart("out", *out, names[i], w.zero, false);
  }
  if (H > 1 << 16 || I > 1 << 16 || Is > 1 << 16) bad("hidden and intermediate sizes are at most 65536");
  l.hidden = (int32_t)H, l.intermediate = (int32_t)I, l.num_experts = (int32_t)E, l.topk = (int32_t)ids.size(1);
  l.shared_intermediate = (int32_t)Is;
  const float limit = (float)number(a[4]);
  l.swiglu_limit = limit == INFINITY ? 0.f : limit;  // (both are no limit, as in MoKConfig; the C ABI takes 0)
  if (out) {
    check("out", *out, x, {kBf16}), shaped("out", *out, x.sizes()), dense("out", *out);
    apart("out", *out, "x", &x, false), apart("out", *out, "router_weights", &rw, false), apart("out", *out, "top_experts", &ids, false);
  }
  const void *px = dense("x", x), *prw = dense("router_weights", rw), *pid = dense("top_experts", ids);
  Tensor y = out ? *out : make({T, H}, x, kBf16);
  const size_t bytes = f_forward_w4_scratch_bytes(&l, T);
  Tensor scratch = make({(int64_t)bytes}, x, kU8);
  const mok_status st = f_forward_w4(&l, px, (const float*)prw, (const int64_t*)pid, T, y.data_ptr(), scratch.data_ptr(), bytes, stream_of(a[6]));
  if (ran(st)) written(out);
  return result(st, {y});
}

// bind(addresses of the C ABI's functions, in the order below)
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
  count("bind", n, 16);
  f_rms_norm = (decltype(f_rms_norm))stream_of(a[0]);
  f_rms_norm_scratch_bytes = (decltype(f_rms_norm_scratch_bytes))stream_of(a[1]);
  f_rms_norm_backward = (decltype(f_rms_norm_backward))stream_of(a[2]);
  f_router_scratch_bytes = (decltype(f_router_scratch_bytes))stream_of(a[3]);
  f_router_topk = (decltype(f_router_topk))stream_of(a[4]);
  f_router_topk_backward = (decltype(f_router_topk_backward))stream_of(a[5]);
  f_adamw_step = (decltype(f_adamw_step))stream_of(a[6]);
  f_grouped_matmul_scratch_bytes = (decltype(f_grouped_matmul_scratch_bytes))stream_of(a[7]);
  f_grouped_matmul = (decltype(f_grouped_matmul))stream_of(a[8]);
  f_grouped_matmul_dx = (decltype(f_grouped_matmul_dx))stream_of(a[9]);
  f_grouped_matmul_dw = (decltype(f_grouped_matmul_dw))stream_of(a[10]);
  f_w4_quantize = (decltype(f_w4_quantize))stream_of(a[11]);
  f_w4_dequantize = (decltype(f_w4_dequantize))stream_of(a[12]);
  f_w4_matmul = (decltype(f_w4_matmul))stream_of(a[13]);
  f_forward_w4_scratch_bytes = (decltype(f_forward_w4_scratch_bytes))stream_of(a[14]);
  f_forward_w4 = (decltype(f_forward_w4))stream_of(a[15]);
  Py_RETURN_NONE;
}

// No C++ exception crosses into the interpreter.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(a, n);
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef method(const char* name) {
  return {name, (PyCFunction)(void (*)(void))guarded<F>, METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind>("bind"),
                         method<rms_norm>("rms_norm"),
                         method<rms_norm_mxfp8>("rms_norm_mxfp8"),
                         method<rms_norm_backward>("rms_norm_backward"),
                         method<router_topk>("router_topk"),
                         method<router_topk_backward>("router_topk_backward"),
                         method<adamw_step>("adamw_step"),
                         method<grouped_matmul>("grouped_matmul"),
                         method<grouped_matmul_backward>("grouped_matmul_backward"),
                         method<w4_quantize>("w4_quantize"),
                         method<w4_dequantize>("w4_dequantize"),
                         method<w4_matmul>("w4_matmul"),
                         method<forward_w4>("forward_w4"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops() { return PyModule_Create(&module_def); }
