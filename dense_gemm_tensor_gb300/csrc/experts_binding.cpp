// Python binding of the mixture-of-experts operators (the module `_experts`
// behind experts.py): checks torch tensors, allocates the outputs and the
// scratch and calls the C entry points of dgt_experts.h.
//
// It is compiled because these operators are a few microseconds long: the same
// marshalling in Python took 12-15 us a call on a GB300's host (an 18 us norm of
// one row whose kernel runs 2.3 us), most of it attribute reads and
// allocations. The entry points' addresses come from the library that
// gemm.load() opened, so there is one copy of the library in the process.
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <limits>
#include <string>

#include "dgt_experts.h"

namespace {

// A refused argument: the Python exception's type and text.
struct Refused {
  PyObject* type;
  std::string text;
};
[[noreturn]] void type_error(const std::string& text) { throw Refused{PyExc_TypeError, text}; }
[[noreturn]] void value_error(const std::string& text) { throw Refused{PyExc_ValueError, text}; }

// The entry points, in the order of kNames.
struct Entries {
  decltype(&gemm_rmsnorm) rmsnorm;
  decltype(&gemm_rmsnorm_backward) rmsnorm_backward;
  decltype(&gemm_rmsnorm_backward_workspace) rmsnorm_backward_workspace;
  decltype(&gemm_route) route;
  decltype(&gemm_route_workspace) route_workspace;
  decltype(&gemm_route_backward) route_backward;
  decltype(&gemm_f16_grouped) f16_grouped;
  decltype(&gemm_bf16_grouped) bf16_grouped;
  decltype(&gemm_e4m3_grouped) e4m3_grouped;
  decltype(&gemm_grouped_rows_workspace) grouped_rows_workspace;
  decltype(&gemm_grouped_weights_workspace) grouped_weights_workspace;
  decltype(&gemm_f16_grouped_wgrad) f16_grouped_wgrad;
  decltype(&gemm_bf16_grouped_wgrad) bf16_grouped_wgrad;
  decltype(&gemm_grouped_wgrad_rows_workspace) grouped_wgrad_rows_workspace;
  decltype(&gemm_combine) combine;
  decltype(&gemm_combine_backward) combine_backward;
};
constexpr const char* kNames[] = {
    "gemm_rmsnorm",          "gemm_rmsnorm_backward", "gemm_rmsnorm_backward_workspace", "gemm_route",
    "gemm_route_workspace",  "gemm_route_backward",   "gemm_f16_grouped",                "gemm_bf16_grouped",
    "gemm_e4m3_grouped",     "gemm_grouped_rows_workspace", "gemm_grouped_weights_workspace", "gemm_f16_grouped_wgrad",         "gemm_bf16_grouped_wgrad",
    "gemm_grouped_wgrad_rows_workspace", "gemm_combine",   "gemm_combine_backward"};
constexpr int kEntries = sizeof(kNames) / sizeof(kNames[0]);
static_assert(sizeof(Entries) == kEntries * sizeof(void*), "one address for each name");
union {
  void* address[kEntries];
  Entries c;
} entry = {};

using Tensor = at::Tensor;

const Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) type_error(std::string(what) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

// The library's number of an element type; -1 for another.
int kind(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kHalf: return GEMM_TYPE_F16;
    case at::kBFloat16: return GEMM_TYPE_BF16;
    case at::kFloat: return GEMM_TYPE_F32;
    case at::kFloat8_e4m3fn: return GEMM_TYPE_E4M3;
    default: return -1;
  }
}
int float_kind(const Tensor& t, const char* what) {
  const int k = kind(t);
  if (k < 0 || k == GEMM_TYPE_E4M3) type_error(std::string(what) + " must be float16, bfloat16 or float32");
  return k;
}

void same_type(const Tensor& t, at::ScalarType dt, const char* what) {
  if (t.scalar_type() != dt) type_error(std::string(what) + " must be " + c10::toString(dt));
}

// Leading dimension of a 2-D CUDA tensor with contiguous rows.
int64_t matrix(const Tensor& t, const char* what) {
  if (t.dim() != 2 || !t.is_cuda()) value_error(std::string(what) + " must be a 2-D CUDA tensor");
  const int64_t rows = t.size(0), cols = t.size(1);
  if (cols > 1 && t.stride(1) != 1) value_error(std::string(what) + " must have unit stride along its rows");
  if (rows <= 1) return cols;
  if (t.stride(0) < cols) value_error(std::string(what) + " must not have rows that overlap");
  return t.stride(0);
}
int64_t matrix(const Tensor& t, const char* what, at::ScalarType dt, int64_t rows, int64_t cols) {
  same_type(t, dt, what);
  const int64_t ld = matrix(t, what);
  if (t.size(0) != rows || t.size(1) != cols)
    value_error(std::string(what) + " must be " + std::to_string(rows) + " x " + std::to_string(cols));
  return ld;
}

// Address of a contiguous CUDA tensor of n elements.
template <class T>
T* vector(const Tensor& t, const char* what, at::ScalarType dt, int64_t n) {
  same_type(t, dt, what);
  if (t.numel() != n || !t.is_cuda() || !t.is_contiguous())
    value_error(std::string(what) + " must be a contiguous CUDA tensor of " + std::to_string(n) + " elements");
  return static_cast<T*>(t.data_ptr());
}
template <class T>
T* vector_or_null(PyObject* o, const char* what, at::ScalarType dt, int64_t n) {
  return o == Py_None ? nullptr : vector<T>(tensor(o, what), what, dt, n);
}

// groups x rows x cols with contiguous rows: leading dimension and matrix stride.
struct Stack {
  int64_t ld, stride;
};
Stack stack(const Tensor& t, const char* what) {
  if (t.dim() != 3 || !t.is_cuda()) value_error(std::string(what) + " must be a 3-D CUDA tensor");
  const int64_t g = t.size(0), r = t.size(1), c = t.size(2);
  if (c > 1 && t.stride(2) != 1) value_error(std::string(what) + " must have unit stride along its rows");
  const int64_t ld = r > 1 ? t.stride(1) : c;
  return {ld, g > 1 ? t.stride(0) : r * ld};
}

Tensor make(at::IntArrayRef size, const Tensor& like, at::ScalarType dt) {
  return at::empty(size, at::TensorOptions().dtype(dt).device(like.device()));
}

// A scratch buffer of n bytes, or nothing.
Tensor scratch(int64_t n, const Tensor& like) { return n > 0 ? make({n}, like, at::kByte) : Tensor(); }

void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

int64_t whole(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
// A whole number that the C call takes as an int.
int whole_int(PyObject* o, const char* what) {
  const int64_t v = whole(o);
  if (v != static_cast<int>(v)) value_error(std::string(what) + " does not fit 32 bits");
  return static_cast<int>(v);
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
template <class... T>
PyObject* tuple_of(const T&... t) {
  PyObject* out = PyTuple_New(sizeof...(T));
  if (out == nullptr) throw python_error();
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(out, i++, wrap(t)), ...);
  return out;
}

// rms_norm(x, weight, residual, eps, 8-bit rows, h_out) -> (y, h, rstd, scale)
PyObject* rms_norm(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const int code = float_kind(x, "x");
  const at::ScalarType dt = x.scalar_type();
  const int64_t ldx = matrix(x, "x"), rows = x.size(0), cols = x.size(1);
  const void* w = vector<void>(tensor(a[1], "weight"), "weight", dt, cols);
  const bool q8 = a[4] == Py_True;
  Tensor h = x;
  const void* residual = nullptr;
  void* ph = nullptr;
  int64_t ldr = 0, ldh = 0;
  if (a[2] != Py_None) {
    const Tensor& r = tensor(a[2], "residual");
    ldr = matrix(r, "residual", dt, rows, cols);
    residual = r.data_ptr();
    if (a[5] != Py_None) {
      h = tensor(a[5], "h_out");
      ldh = matrix(h, "h_out", dt, rows, cols);
    } else {
      h = make({rows, cols}, x, dt);
      ldh = cols;
    }
    ph = h.data_ptr();
  }
  Tensor y = make({rows, cols}, x, q8 ? at::kFloat8_e4m3fn : dt), rstd = make({rows}, x, at::kFloat);
  Tensor scale = q8 ? make({rows}, x, at::kFloat) : Tensor();
  if (cols == 0) {  // the call writes nothing: the mean of no elements, and the least scale
    rstd.fill_(std::numeric_limits<double>::quiet_NaN());
    if (q8) scale.fill_(1e-12 / 448);
  }
  const int st = entry.c.rmsnorm(code, rows, cols, x.data_ptr(), ldx, residual, ldr, w, static_cast<float>(real(a[3])), ph,
                                 ldh, q8 ? GEMM_TYPE_E4M3 : code, y.data_ptr(), cols,
                                 q8 ? static_cast<float*>(scale.data_ptr()) : nullptr,
                                 static_cast<float*>(rstd.data_ptr()), stream_of(x));
  return st != GEMM_OK ? PyLong_FromLong(st) : tuple_of(y, h, rstd, scale);
}

// rms_norm_backward(dy, h, weight, rstd, dh) -> (dx, dweight)
PyObject* rms_norm_backward(PyObject* const* a) {
  const Tensor &dy = tensor(a[0], "dy"), &h = tensor(a[1], "h");
  const int code = float_kind(h, "h");
  const at::ScalarType dt = h.scalar_type();
  const int64_t ldh = matrix(h, "h"), rows = h.size(0), cols = h.size(1);
  const int64_t lddy = matrix(dy, "dy", dt, rows, cols);
  const void* w = vector<void>(tensor(a[2], "weight"), "weight", dt, cols);
  const float* rstd = vector<float>(tensor(a[3], "rstd"), "rstd", at::kFloat, rows);
  const void* dh = nullptr;
  int64_t lddh = 0;
  if (a[4] != Py_None) {
    const Tensor& t = tensor(a[4], "dh");
    lddh = matrix(t, "dh", dt, rows, cols);
    dh = t.data_ptr();
  }
  Tensor dx = make({rows, cols}, h, dt), dw = make({cols}, h, dt);
  const int64_t need = entry.c.rmsnorm_backward_workspace(rows, cols);
  Tensor ws = scratch(need, h);
  const int st = entry.c.rmsnorm_backward(code, rows, cols, dy.data_ptr(), lddy, h.data_ptr(), ldh, w, rstd, dh, lddh,
                                          dx.data_ptr(), cols, dw.data_ptr(), need > 0 ? ws.data_ptr() : nullptr, need,
                                          stream_of(h));
  return st != GEMM_OK ? PyLong_FromLong(st) : tuple_of(dx, dw);
}

gemm_route_config_t route_config(PyObject* k, PyObject* score, PyObject* groups, PyObject* kept, PyObject* renormalize,
                                 PyObject* scale) {
  return {whole_int(k, "k"),       whole_int(score, "score"), whole_int(groups, "groups"), whole_int(kept, "kept_groups"),
          truth(renormalize), static_cast<float>(real(scale))};
}

// route(logits, k, score, bias, groups, kept_groups, renormalize, scale) -> (ids, weights, slots, rows, offsets)
PyObject* route(PyObject* const* a) {
  const Tensor& logits = tensor(a[0], "logits");
  const int code = float_kind(logits, "logits");
  const int64_t ld = matrix(logits, "logits"), tokens = logits.size(0), experts = logits.size(1);
  const gemm_route_config_t cfg = route_config(a[1], a[2], a[4], a[5], a[6], a[7]);
  const float* bias = vector_or_null<float>(a[3], "bias", at::kFloat, experts);
  const int64_t k = cfg.k > 0 && cfg.k <= experts ? cfg.k : 0;  // (the call refuses others)
  Tensor ids = make({tokens, k}, logits, at::kInt), weights = make({tokens, k}, logits, at::kFloat);
  Tensor slots = make({tokens, k}, logits, at::kInt), rows = make({tokens * k}, logits, at::kInt);
  Tensor offsets = make({experts + 1}, logits, at::kInt);
  const int e = experts > (1 << 30) ? 1 << 30 : static_cast<int>(experts);
  const int64_t need = entry.c.route_workspace(tokens, e, cfg.k);
  Tensor ws = scratch(need, logits);
  auto i32 = [](const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); };
  const int st = entry.c.route(code, tokens, e, logits.data_ptr(), ld, bias, &cfg, i32(ids),
                               static_cast<float*>(weights.data_ptr()), i32(slots), i32(rows), i32(offsets),
                               need > 0 ? ws.data_ptr() : nullptr, need, stream_of(logits));
  return st != GEMM_OK ? PyLong_FromLong(st) : tuple_of(ids, weights, slots, rows, offsets);
}

// route_backward(dweights, logits, ids, score, renormalize, scale) -> (dlogits,)
PyObject* route_backward(PyObject* const* a) {
  const Tensor &logits = tensor(a[1], "logits"), &ids = tensor(a[2], "ids");
  const int code = float_kind(logits, "logits");
  const int64_t ld = matrix(logits, "logits"), tokens = logits.size(0), experts = logits.size(1);
  if (ids.dim() != 2 || ids.size(0) != tokens) value_error("ids must be T x k");
  const int64_t k = ids.size(1);
  gemm_route_config_t cfg = {static_cast<int>(k > 1 << 20 ? 1 << 20 : k), whole_int(a[3], "score"), 1, 1, truth(a[4]),
                             static_cast<float>(real(a[5]))};
  const int32_t* i = vector<int32_t>(ids, "ids", at::kInt, tokens * k);
  const float* d = vector<float>(tensor(a[0], "dweights"), "dweights", at::kFloat, tokens * k);
  Tensor out = make({tokens, experts}, logits, logits.scalar_type());
  const int st = entry.c.route_backward(code, tokens, experts > (1 << 30) ? 1 << 30 : static_cast<int>(experts),
                                        logits.data_ptr(), ld, i, d, &cfg, out.data_ptr(), experts, stream_of(logits));
  return st != GEMM_OK ? PyLong_FromLong(st) : tuple_of(out);
}

// expert_matmul(A, W, offsets, rows, layout, out, alpha, a_scale, w_scale, bias, activation) -> (C,)
PyObject* expert_matmul(PyObject* const* a) {
  const Tensor &A = tensor(a[0], "A"), &W = tensor(a[1], "W");
  const at::ScalarType dt = A.scalar_type();
  const int code = kind(A);
  if (code < 0 || code == GEMM_TYPE_F32) type_error("A must be float16, bfloat16 or float8_e4m3fn");
  if (W.scalar_type() != dt) type_error("A and W must have the same dtype");
  const int64_t lda = matrix(A, "A"), a_rows = A.size(0), K = A.size(1);
  const Stack w = stack(W, "W");
  const int layout = whole_int(a[4], "layout");
  const bool kmajor = layout == GEMM_B_K_MAJOR;
  const int64_t experts = W.size(0), N = W.size(kmajor ? 1 : 2);
  if (W.size(kmajor ? 2 : 1) != K) value_error("W's K dimension does not match A");
  const at::ScalarType out_dt = code == GEMM_TYPE_E4M3 ? at::kBFloat16 : dt;
  const int32_t* offsets = vector<int32_t>(tensor(a[2], "offsets"), "offsets", at::kInt, experts + 1);
  const int e = experts > (1 << 30) ? 1 << 30 : static_cast<int>(experts);
  int64_t slots = a_rows;
  const int32_t* rows = nullptr;
  if (a[3] != Py_None) {
    const Tensor& r = tensor(a[3], "rows");
    slots = r.numel();
    rows = vector<int32_t>(r, "rows", at::kInt, slots);
  }
  const int act = whole_int(a[10], "activation");
  const int64_t need = entry.c.grouped_rows_workspace(code, e, slots, K, a_rows, lda, rows != nullptr) +
                       entry.c.grouped_weights_workspace(code, e, N, K, w.ld, w.stride, layout, act);
  const int64_t cols = act == GEMM_ACT_SILU_GATED ? N / 2 : N;
  Tensor out;
  int64_t ldc = cols;
  if (a[5] != Py_None) {
    out = tensor(a[5], "out");
    ldc = matrix(out, "out", out_dt, slots, cols);
  } else {
    out = make({slots, cols}, A, out_dt);
  }
  Tensor ws = scratch(need, A);
  gemm_grouped_epilogue_t epi;
  epi.alpha = static_cast<float>(real(a[6]));
  epi.row_scale = vector_or_null<float>(a[7], "a_scale", at::kFloat, a_rows);
  epi.col_scale = vector_or_null<float>(a[8], "w_scale", at::kFloat, experts * N);
  epi.bias = vector_or_null<void>(a[9], "bias", out_dt, experts * N);
  epi.activation = act;
  void* wp = need > 0 ? ws.data_ptr() : nullptr;
  void* s = stream_of(A);
  int st;
  if (code == GEMM_TYPE_E4M3) {
    st = entry.c.e4m3_grouped(e, offsets, slots, N, K, static_cast<const uint8_t*>(A.data_ptr()), a_rows, lda, rows,
                              static_cast<const uint8_t*>(W.data_ptr()), w.ld, w.stride,
                              static_cast<uint16_t*>(out.data_ptr()), ldc, layout, &epi, wp, need, s);
  } else {
    const auto fn = code == GEMM_TYPE_F16 ? entry.c.f16_grouped : entry.c.bf16_grouped;
    st = fn(e, offsets, slots, N, K, static_cast<const uint16_t*>(A.data_ptr()), a_rows, lda, rows,
            static_cast<const uint16_t*>(W.data_ptr()), w.ld, w.stride, static_cast<uint16_t*>(out.data_ptr()), ldc,
            layout, &epi, wp, need, s);
  }
  return st != GEMM_OK ? PyLong_FromLong(st) : tuple_of(out);
}

// expert_weight_grad(A, dC, offsets, rows, layout, out) -> (dW,)
PyObject* expert_weight_grad(PyObject* const* a) {
  const Tensor &A = tensor(a[0], "A"), &dC = tensor(a[1], "dC"), &off = tensor(a[2], "offsets");
  const at::ScalarType dt = A.scalar_type();
  if (dt != at::kHalf && dt != at::kBFloat16) type_error("A must be float16 or bfloat16");
  const int64_t lda = matrix(A, "A"), a_rows = A.size(0), K = A.size(1);
  int64_t slots = a_rows;
  const int32_t* rows = nullptr;
  if (a[3] != Py_None) {
    const Tensor& r = tensor(a[3], "rows");
    slots = r.numel();
    rows = vector<int32_t>(r, "rows", at::kInt, slots);
  }
  same_type(dC, dt, "dC");
  const int64_t lddc = matrix(dC, "dC"), N = dC.size(1);
  if (dC.size(0) != slots) value_error("dC must have one row per slot");
  const int64_t experts = off.numel() - 1;
  const int32_t* offsets = vector<int32_t>(off, "offsets", at::kInt, experts + 1);
  const int e = experts > (1 << 30) ? 1 << 30 : static_cast<int>(experts);
  const int layout = whole_int(a[4], "layout");
  const int64_t r0 = layout == GEMM_B_K_MAJOR ? N : K, r1 = layout == GEMM_B_K_MAJOR ? K : N;
  Tensor out;
  if (a[5] != Py_None) {
    out = tensor(a[5], "out");
    same_type(out, dt, "out");
    if (out.dim() != 3 || out.size(0) != experts || out.size(1) != r0 || out.size(2) != r1)
      value_error("out must be " + std::to_string(experts) + " x " + std::to_string(r0) + " x " + std::to_string(r1));
  } else {
    out = make({experts < 0 ? 0 : experts, r0, r1}, A, dt);
  }
  const Stack w = stack(out, "out");
  const int64_t need = entry.c.grouped_wgrad_rows_workspace(e, slots, N, K, a_rows, lda, rows != nullptr, lddc);
  Tensor ws = scratch(need, A);
  const auto fn = dt == at::kHalf ? entry.c.f16_grouped_wgrad : entry.c.bf16_grouped_wgrad;
  const int st = fn(e, offsets, slots, N, K, static_cast<const uint16_t*>(A.data_ptr()), a_rows, lda, rows,
                    static_cast<const uint16_t*>(dC.data_ptr()), lddc, static_cast<uint16_t*>(out.data_ptr()), w.ld,
                    w.stride, layout, need > 0 ? ws.data_ptr() : nullptr, need, stream_of(A));
  return st != GEMM_OK ? PyLong_FromLong(st) : tuple_of(out);
}

// combine(z, slots, weights, residual, out) -> (y,)
PyObject* combine(PyObject* const* a) {
  const Tensor &z = tensor(a[0], "z"), &slots = tensor(a[1], "slots");
  const int code = float_kind(z, "z");
  const at::ScalarType dt = z.scalar_type();
  const int64_t ldz = matrix(z, "z"), nslots = z.size(0), cols = z.size(1);
  if (slots.dim() != 2) value_error("slots must be T x k");
  const int64_t tokens = slots.size(0), k = slots.size(1);
  const int32_t* i = vector<int32_t>(slots, "slots", at::kInt, tokens * k);
  const float* w = vector_or_null<float>(a[2], "weights", at::kFloat, tokens * k);
  const void* residual = nullptr;
  int64_t ldr = 0, ldy = cols;
  if (a[3] != Py_None) {
    const Tensor& r = tensor(a[3], "residual");
    ldr = matrix(r, "residual", dt, tokens, cols);
    residual = r.data_ptr();
  }
  Tensor out;
  if (a[4] != Py_None) {
    out = tensor(a[4], "out");
    ldy = matrix(out, "out", dt, tokens, cols);
  } else {
    out = make({tokens, cols}, z, dt);
  }
  const int st = entry.c.combine(code, tokens, cols, static_cast<int>(k > 1 << 20 ? 1 << 20 : k), z.data_ptr(), ldz, nslots,
                                 i, w, residual, ldr, out.data_ptr(), ldy, stream_of(z));
  return st != GEMM_OK ? PyLong_FromLong(st) : tuple_of(out);
}

// combine_backward(dy, z, slots, weights, offsets) -> (dz, dweights)
PyObject* combine_backward(PyObject* const* a) {
  const Tensor &dy = tensor(a[0], "dy"), &z = tensor(a[1], "z"), &slots = tensor(a[2], "slots");
  const int code = float_kind(z, "z");
  const at::ScalarType dt = z.scalar_type();
  const int64_t ldz = matrix(z, "z"), nslots = z.size(0), cols = z.size(1);
  if (slots.dim() != 2) value_error("slots must be T x k");
  const int64_t tokens = slots.size(0), k = slots.size(1);
  const int64_t lddy = matrix(dy, "dy", dt, tokens, cols);
  const int32_t* i = vector<int32_t>(slots, "slots", at::kInt, tokens * k);
  const float* w = vector_or_null<float>(a[3], "weights", at::kFloat, tokens * k);
  const int32_t* used = nullptr;
  if (a[4] != Py_None) {
    const Tensor& off = tensor(a[4], "offsets");
    if (off.numel() < 1) value_error("offsets must not be empty");
    used = vector<int32_t>(off, "offsets", at::kInt, off.numel()) + off.numel() - 1;
  }
  // (by the argument, not by w: the address of no weights is null too)
  const bool weighted = a[3] != Py_None;
  Tensor dz = make({nslots, cols}, z, dt), dw = weighted ? make({tokens, k}, z, at::kFloat) : Tensor();
  const int st = entry.c.combine_backward(code, tokens, cols, static_cast<int>(k > 1 << 20 ? 1 << 20 : k), dy.data_ptr(),
                                          lddy, z.data_ptr(), ldz, nslots, i, w, used, dz.data_ptr(), cols,
                                          weighted ? static_cast<float*>(dw.data_ptr()) : nullptr, stream_of(z));
  return st != GEMM_OK ? PyLong_FromLong(st) : tuple_of(dz, dw);
}

// The Python-callable form: N arguments, and every C++ exception as a Python one.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* method(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are taken, %zd were given", N, n);
    return nullptr;
  }
  if (entry.address[0] == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "bind() has not given the library's entry points");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// bind({name: address}): the entry points of the loaded library.
PyObject* bind(PyObject*, PyObject* addresses) {
  void* found[kEntries];
  for (int i = 0; i < kEntries; ++i) {
    PyObject* v = PyDict_Check(addresses) ? PyDict_GetItemString(addresses, kNames[i]) : nullptr;
    found[i] = v != nullptr ? PyLong_AsVoidPtr(v) : nullptr;
    if (found[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "no address of %s", kNames[i]);
      return nullptr;
    }
  }
  for (int i = 0; i < kEntries; ++i) entry.address[i] = found[i];
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef def(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&method<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         def<rms_norm, 6>("rms_norm"),
                         def<rms_norm_backward, 5>("rms_norm_backward"),
                         def<route, 8>("route"),
                         def<route_backward, 6>("route_backward"),
                         def<expert_matmul, 11>("expert_matmul"),
                         def<expert_weight_grad, 6>("expert_weight_grad"),
                         def<combine, 5>("combine"),
                         def<combine_backward, 5>("combine_backward"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_experts", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__experts(void) { return PyModule_Create(&module); }
