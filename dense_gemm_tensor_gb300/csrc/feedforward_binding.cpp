// Python binding of the feed-forward operators (the module `_feedforward` behind
// feedforward.py): checks torch tensors, allocates the outputs and the scratch and
// calls the C entry points of dgt_feedforward.h. Compiled for the reason that
// experts_binding.cpp gives: the marshalling in Python takes longer than the
// smallest kernels.
#include "binding.h"
#include "dgt_feedforward.h"

namespace {

// The entry points, in the order of kNames.
struct Entries {
  decltype(&gemm_layernorm) layernorm;
  decltype(&gemm_layernorm_backward) layernorm_backward;
  decltype(&gemm_layernorm_backward_workspace) layernorm_backward_workspace;
  decltype(&gemm_gated) gated;
  decltype(&gemm_gated_workspace) gated_workspace;
  decltype(&gemm_gated_backward) gated_backward;
  decltype(&gemm_gated_backward_workspace) gated_backward_workspace;
  decltype(&gemm_e4m3_blocks) e4m3_blocks;
  decltype(&gemm_quantize_blocks) quantize_blocks;
};
constexpr const char* kNames[] = {"gemm_layernorm",       "gemm_layernorm_backward",
                                  "gemm_layernorm_backward_workspace", "gemm_gated",
                                  "gemm_gated_workspace", "gemm_gated_backward",
                                  "gemm_gated_backward_workspace",     "gemm_e4m3_blocks",
                                  "gemm_quantize_blocks"};
constexpr int kEntries = sizeof(kNames) / sizeof(kNames[0]);
static_assert(sizeof(Entries) == kEntries * sizeof(void*), "one address for each name");
union {
  void* address[kEntries];
  Entries c;
} entry = {};

constexpr int64_t kBlock = 128;

// Every tensor of a call is on one device.
void same_device(const Tensor& t, const Tensor& like, const char* what) {
  if (t.device() != like.device()) value_error(std::string(what) + " is on another device");
}
// The current device is the one that the library launches on.
void current_device(const Tensor& t, const char* what) {
  if (t.is_cuda() && t.device().index() != c10::cuda::current_device())
    value_error(std::string(what) + " is not on the current CUDA device");
}

// A matrix (or nothing): address and leading dimension.
struct Matrix {
  void* p = nullptr;
  int64_t ld = 0;
};
Matrix matrix_or_null(PyObject* o, const char* what, at::ScalarType dt, int64_t rows, int64_t cols, const Tensor& like) {
  Matrix m;
  if (o == Py_None) return m;
  const Tensor& t = tensor(o, what);
  m.ld = matrix(t, what, dt, rows, cols);
  same_device(t, like, what);
  m.p = t.data_ptr();
  return m;
}

template <class T>
T* vector_on(PyObject* o, const char* what, at::ScalarType dt, int64_t n, const Tensor& like) {
  const Tensor& t = tensor(o, what);
  T* p = vector<T>(t, what, dt, n);
  same_device(t, like, what);
  return p;
}

// Part `i` of a buffer of vectors of `n` floats. (An allocation costs twice what another tensor on its memory does.)
Tensor part(const Tensor& buffer, int64_t i, int64_t n) {
  c10::Storage storage = buffer.storage();
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(std::move(storage), buffer.key_set(), buffer.dtype());
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  t.unsafeGetTensorImpl()->set_storage_offset(buffer.storage_offset() + i * n);
  return t;
}

// layer_norm(x, weight, bias, residual, eps, 8-bit rows, h_out) -> (y, h, mean, rstd, scale)
PyObject* layer_norm(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const int code = float_kind(x, "x");
  const at::ScalarType dt = x.scalar_type();
  const int64_t ldx = matrix(x, "x"), rows = x.size(0), cols = x.size(1);
  current_device(x, "x");
  const void* w = vector_on<void>(a[1], "weight", dt, cols, x);
  const void* b = a[2] == Py_None ? nullptr : vector_on<void>(a[2], "bias", dt, cols, x);
  const bool q8 = a[5] == Py_True;
  Tensor h = x;
  void* ph = nullptr;
  int64_t ldh = 0;
  const Matrix residual = matrix_or_null(a[3], "residual", dt, rows, cols, x);
  if (a[3] != Py_None) {
    if (a[6] != Py_None) {
      h = tensor(a[6], "h_out");
      ldh = matrix(h, "h_out", dt, rows, cols);
      same_device(h, x, "h_out");
    } else {
      h = make({rows, cols}, x, dt);
      ldh = cols;
    }
    ph = h.data_ptr();
  } else if (a[6] != Py_None) {
    value_error("h_out is given without a residual: h is x");
  }
  Tensor y = make({rows, cols}, x, q8 ? at::kFloat8_e4m3fn : dt);
  const Tensor vectors = make({(q8 ? 3 : 2) * rows}, x, at::kFloat);
  Tensor mean = part(vectors, 0, rows), rstd = part(vectors, 1, rows), scale = q8 ? part(vectors, 2, rows) : Tensor();
  if (cols == 0) {  // the call writes nothing: the mean of no elements, and the least scale
    mean.fill_(std::numeric_limits<double>::quiet_NaN());
    rstd.fill_(std::numeric_limits<double>::quiet_NaN());
    if (q8) scale.fill_(1e-12 / 448);
  }
  const int st = entry.c.layernorm(code, rows, cols, x.data_ptr(), ldx, residual.p, residual.ld, w, b,
                                   static_cast<float>(real(a[4])), ph, ldh, q8 ? GEMM_TYPE_E4M3 : code, y.data_ptr(), cols,
                                   q8 ? static_cast<float*>(scale.data_ptr()) : nullptr,
                                   static_cast<float*>(mean.data_ptr()), static_cast<float*>(rstd.data_ptr()), stream_of(x));
  return st != GEMM_OK ? PyLong_FromLong(st) : tuple_of(y, h, mean, rstd, scale);
}

// layer_norm_backward(dy, h, weight, mean, rstd, dh) -> (dx, dweight, dbias)
PyObject* layer_norm_backward(PyObject* const* a) {
  const Tensor& h = tensor(a[1], "h");
  const int code = float_kind(h, "h");
  const at::ScalarType dt = h.scalar_type();
  const int64_t ldh = matrix(h, "h"), rows = h.size(0), cols = h.size(1);
  current_device(h, "h");
  if (a[0] == Py_None) type_error("dy must be a torch.Tensor");
  const Matrix dy = matrix_or_null(a[0], "dy", dt, rows, cols, h), dh = matrix_or_null(a[5], "dh", dt, rows, cols, h);
  const void* w = vector_on<void>(a[2], "weight", dt, cols, h);
  const float* mean = vector_on<float>(a[3], "mean", at::kFloat, rows, h);
  const float* rstd = vector_on<float>(a[4], "rstd", at::kFloat, rows, h);
  Tensor dx = make({rows, cols}, h, dt), dw = make({cols}, h, dt), db = make({cols}, h, dt);
  const int64_t need = entry.c.layernorm_backward_workspace(rows, cols);
  Tensor ws = scratch(need, h);
  const int st = entry.c.layernorm_backward(code, rows, cols, dy.p, dy.ld, h.data_ptr(), ldh, w, mean, rstd, dh.p, dh.ld,
                                            dx.data_ptr(), cols, dw.data_ptr(), db.data_ptr(),
                                            need > 0 ? ws.data_ptr() : nullptr, need, stream_of(h));
  return st != GEMM_OK ? PyLong_FromLong(st) : tuple_of(dx, dw, db);
}

// A gated product's operands.
struct Gated {
  int code, layout;
  at::ScalarType dt;
  int64_t M, K, F, lda, ldw;
};
Gated gated_operands(const Tensor& A, const Tensor& W, PyObject* layout) {
  Gated g;
  g.code = kind(A);
  g.dt = A.scalar_type();
  if (g.code != GEMM_TYPE_F16 && g.code != GEMM_TYPE_BF16) type_error("A must be float16 or bfloat16");
  if (W.scalar_type() != g.dt) type_error("A and W must have the same dtype");
  g.lda = matrix(A, "A");
  g.ldw = matrix(W, "W");
  current_device(A, "A");
  same_device(W, A, "W");
  g.layout = whole_int(layout, "layout");
  const bool km = g.layout == GEMM_B_K_MAJOR;
  g.M = A.size(0);
  g.K = A.size(1);
  if (W.size(km ? 1 : 0) != g.K) value_error("W's K dimension does not match A");
  if (W.size(km ? 0 : 1) % 2 != 0) value_error("W must hold a gate and a value half of the same width");
  g.F = W.size(km ? 0 : 1) / 2;
  return g;
}

// gated_matmul(A, W, layout, activation, bias, keep, out) -> (c, up)
PyObject* gated_matmul(PyObject* const* a) {
  const Tensor &A = tensor(a[0], "A"), &W = tensor(a[1], "W");
  const Gated g = gated_operands(A, W, a[2]);
  const void* bias = a[4] == Py_None ? nullptr : vector_on<void>(a[4], "bias", g.dt, 2 * g.F, A);
  const bool keep = truth(a[5]);
  Tensor c, up;
  int64_t ldc = g.F, ldup = 2 * g.F;
  if (a[6] != Py_None) {
    c = tensor(a[6], "out");
    ldc = matrix(c, "out", g.dt, g.M, g.F);
    same_device(c, A, "out");
  } else {
    c = make({g.M, g.F}, A, g.dt);
  }
  if (keep) up = make({g.M, 2 * g.F}, A, g.dt);
  const int64_t need = entry.c.gated_workspace(g.code, g.M, g.F, g.K, g.lda, g.ldw, g.layout);
  Tensor ws = scratch(need, A);
  const int st = entry.c.gated(g.code, g.M, g.F, g.K, A.data_ptr(), g.lda, W.data_ptr(), g.ldw, g.layout,
                               whole_int(a[3], "activation"), bias, c.data_ptr(), ldc, keep ? up.data_ptr() : nullptr, ldup,
                               need > 0 ? ws.data_ptr() : nullptr, need, stream_of(A));
  return st != GEMM_OK ? PyLong_FromLong(st) : tuple_of(c, up);
}

// gated_matmul_backward(dC, A, W, up, layout, activation, want dA, want dW, want dbias) -> (dA, dW, dbias)
PyObject* gated_matmul_backward(PyObject* const* a) {
  const Tensor &A = tensor(a[1], "A"), &W = tensor(a[2], "W");
  const Gated g = gated_operands(A, W, a[4]);
  if (a[0] == Py_None || a[3] == Py_None) type_error("dC and up must be torch.Tensors");
  const Matrix dc = matrix_or_null(a[0], "dC", g.dt, g.M, g.F, A), up = matrix_or_null(a[3], "up", g.dt, g.M, 2 * g.F, A);
  const bool da = truth(a[6]), dw = truth(a[7]), db = truth(a[8]);
  const bool km = g.layout == GEMM_B_K_MAJOR;
  const int64_t w_rows = km ? 2 * g.F : g.K, w_cols = km ? g.K : 2 * g.F;
  Tensor dA = da ? make({g.M, g.K}, A, g.dt) : Tensor(), dW = dw ? make({w_rows, w_cols}, A, g.dt) : Tensor();
  Tensor dbias = db ? make({2 * g.F}, A, g.dt) : Tensor();
  const int64_t need = entry.c.gated_backward_workspace(g.code, g.M, g.F, g.K, g.lda, g.ldw, g.layout, da, dw, db);
  Tensor ws = scratch(need, A);
  const int st = entry.c.gated_backward(g.code, g.M, g.F, g.K, dc.p, dc.ld, up.p, up.ld, A.data_ptr(), g.lda, W.data_ptr(),
                                        g.ldw, g.layout, whole_int(a[5], "activation"), da ? dA.data_ptr() : nullptr, g.K,
                                        dw ? dW.data_ptr() : nullptr, w_cols, db ? dbias.data_ptr() : nullptr,
                                        need > 0 ? ws.data_ptr() : nullptr, need, stream_of(A));
  return st != GEMM_OK ? PyLong_FromLong(st) : tuple_of(dA, dW, dbias);
}

// Scales of rows x blocks: any strides that do not run backwards.
struct Scales {
  const float* p;
  int64_t row, block;
};
Scales block_scales(PyObject* o, const char* what, int64_t rows, int64_t blocks, const Tensor& like) {
  const Tensor& t = tensor(o, what);
  same_type(t, at::kFloat, what);
  if (t.dim() != 2 || !t.is_cuda() || t.size(0) != rows || t.size(1) != blocks)
    value_error(std::string(what) + " must be a CUDA tensor of " + std::to_string(rows) + " x " + std::to_string(blocks));
  same_device(t, like, what);
  return {static_cast<const float*>(t.data_ptr()), rows > 1 ? t.stride(0) : 0, blocks > 1 ? t.stride(1) : 0};
}

// matmul_blocks(A, B, a_scale, b_scale, out) -> (C,)
PyObject* matmul_blocks(PyObject* const* a) {
  const Tensor &A = tensor(a[0], "A"), &B = tensor(a[1], "B");
  same_type(A, at::kFloat8_e4m3fn, "A");
  same_type(B, at::kFloat8_e4m3fn, "B");
  const int64_t lda = matrix(A, "A"), ldb = matrix(B, "B"), M = A.size(0), N = B.size(0), K = A.size(1);
  current_device(A, "A");
  same_device(B, A, "B");
  if (B.size(1) != K) value_error("B must be N x K");
  const int64_t blocks = (K + kBlock - 1) / kBlock;
  const Scales sa = block_scales(a[2], "a_scale", M, blocks, A);
  const Tensor& bs = tensor(a[3], "b_scale");
  const int64_t runs = (N + kBlock - 1) / kBlock;
  const bool tall = bs.dim() == 2 && bs.size(0) == runs;  // (N = 1: the same either way)
  const Scales sb = block_scales(a[3], tall || bs.dim() != 2 || bs.size(0) != N ? "b_scale (of 128 x 128 blocks, or N x blocks)" : "b_scale",
                                 tall ? runs : N, blocks, A);
  Tensor out;
  int64_t ldc = N;
  if (a[4] != Py_None) {
    out = tensor(a[4], "out");
    ldc = matrix(out, "out", at::kBFloat16, M, N);
    same_device(out, A, "out");
  } else {
    out = make({M, N}, A, at::kBFloat16);
  }
  const int st = entry.c.e4m3_blocks(M, N, K, static_cast<const uint8_t*>(A.data_ptr()), lda, sa.p, sa.row, sa.block,
                                     static_cast<const uint8_t*>(B.data_ptr()), ldb, sb.p, sb.row, sb.block,
                                     tall ? int(kBlock) : 1, static_cast<uint16_t*>(out.data_ptr()), ldc, stream_of(A));
  return st != GEMM_OK ? PyLong_FromLong(st) : tuple_of(out);
}

// quantize_blocks(x, rows, transpose) -> (q, scale)
PyObject* quantize_blocks(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const int code = float_kind(x, "x");
  const int64_t ldx = matrix(x, "x"), rows = x.size(0), cols = x.size(1);
  current_device(x, "x");
  const int tall = whole_int(a[1], "rows");
  const bool transpose = truth(a[2]);
  const int64_t out_rows = transpose ? cols : rows, out_cols = transpose ? rows : cols;
  const int64_t blocks = (out_cols + kBlock - 1) / kBlock, runs = tall == 1 ? out_rows : (out_rows + kBlock - 1) / kBlock;
  // q's rows start on 16-byte boundaries, as the product wants them; scales of single rows lie block by block
  const int64_t ldq = (out_cols + 15) / 16 * 16, s_row = tall == 1 ? 1 : blocks, s_block = tall == 1 ? runs : 1;
  Tensor q = make_strided({out_rows, out_cols}, {ldq, 1}, x, at::kFloat8_e4m3fn);
  Tensor scale = make_strided({runs, blocks}, {s_row, s_block}, x, at::kFloat);
  const int st = entry.c.quantize_blocks(code, rows, cols, x.data_ptr(), ldx, tall, transpose,
                                         static_cast<uint8_t*>(q.data_ptr()), ldq, static_cast<float*>(scale.data_ptr()),
                                         s_row, s_block, stream_of(x));
  return st != GEMM_OK ? PyLong_FromLong(st) : tuple_of(q, scale);
}

bool is_bound() { return entry.address[0] != nullptr; }

PyObject* bind(PyObject*, PyObject* addresses) { return bind_entries(addresses, kNames, entry.address, kEntries); }

PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         def<layer_norm, 7>("layer_norm"),
                         def<layer_norm_backward, 6>("layer_norm_backward"),
                         def<gated_matmul, 7>("gated_matmul"),
                         def<gated_matmul_backward, 9>("gated_matmul_backward"),
                         def<matmul_blocks, 5>("matmul_blocks"),
                         def<quantize_blocks, 3>("quantize_blocks"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_feedforward", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__feedforward(void) { return PyModule_Create(&module); }
