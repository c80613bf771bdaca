// The MXFP4 operators' and residual_norm's binding, compiled for the same reason
// as the attention operators' and into the same module (attention_binding.cpp):
// one token's calls are short.  The functions take mxfp4.py's arguments by
// position and run on the current stream of their operands' device.
#include <array>

#include "binding.h"

namespace fgg_binding {
namespace {

constexpr at::ScalarType kCodes = at::ScalarType::Float4_e2m1fn_x2, kScales = at::ScalarType::Float8_e8m0fnu;

// Bytes of a format: uint8, or the type that torch has for it.
const Tensor& bytes(PyObject* o, const char* name, at::ScalarType format, int64_t dim) {
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a tensor");
  const Tensor& t = THPVariable_Unpack(o);
  const at::ScalarType d = t.scalar_type();
  TORCH_CHECK_VALUE(d == at::kByte || d == format || (d == at::kChar && format == kCodes), name, " must hold ",
                    format == kCodes ? "packed E2M1 codes (uint8 / float4_e2m1fn_x2)" : "E8M0 codes (uint8 / float8_e8m0fnu)",
                    ", got ", type_name(d));
  TORCH_CHECK_VALUE(t.dim() == dim, name, " must be ", dim, "-D");
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a GPU tensor");
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
  return t;
}

// Codes [..., K / 2] and their scales [..., K / 32]; K.
int64_t pair(const Tensor& codes, const Tensor& scales, const char* name) {
  const int64_t K = 2 * codes.size(-1);
  bool same = codes.get_device() == scales.get_device() && K == 32 * scales.size(-1);
  for (int64_t i = 0; i + 1 < codes.dim(); ++i) same = same && codes.size(i) == scales.size(i);
  TORCH_CHECK_VALUE(same, name, " must have one scale for each 32 codes of a row (16 bytes), on their device: got ",
                    scales.sizes(), " for codes of ", codes.sizes());
  return K;
}

Tensor empty_bytes(at::IntArrayRef sizes, const Tensor& like) { return at::empty(sizes, like.options().dtype(at::kByte)); }

PyObject* both(Tensor a, Tensor b) {
  THPObjectPtr first(THPVariable_Wrap(std::move(a)));
  THPObjectPtr second(THPVariable_Wrap(std::move(b)));
  return PyTuple_Pack(2, first.get(), second.get());
}

// A BF16 [T, H] operand, H contiguous.
const Tensor& rows_of(PyObject* o, const char* name) {
  const Tensor& t = tensor(o, name, at::kBFloat16, 2);
  TORCH_CHECK_VALUE(t.stride(1) == 1 || t.size(1) <= 1, name, " must be contiguous in its last dimension");
  return t;
}

}  // namespace

// X, rows
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 2);
  const Tensor& x = tensor(a[0], "X", at::kBFloat16, 2);
  TORCH_CHECK_VALUE(x.is_contiguous(), "X must be contiguous");
  const c10::DeviceGuard guard(x.device());
  const int64_t T = x.size(0), K = x.size(1);
  const bool expand = a[1] != Py_None;
  const int32_t* map = expand ? vector<int32_t>(a[1], "rows", -1, at::kInt, x) : nullptr;
  const int64_t R = expand ? THPVariable_Unpack(a[1]).size(0) : T;
  TORCH_CHECK_VALUE(K >= 32 && K % 32 == 0, "X must have rows of a multiple of 32 values, got ", K);
  const std::array<int64_t, 2> qs{R, K / 2}, ss{R, K / 32};
  Tensor q = empty_bytes(qs, x), s = empty_bytes(ss, x);
  if (R) {
    const int m = as_int(R, "R"), t = as_int(T, "T"), k = as_int(K, "K");
    void* const stream = stream_on(x);
    call([&] {
      return expand ? quantize_mxfp4_rows(x.const_data_ptr(), map, q.data_ptr(), s.data_ptr(), m, t, k, stream)
                    : quantize_mxfp4(x.const_data_ptr(), q.data_ptr(), s.data_ptr(), m, k, stream);
    });
  }
  return both(std::move(q), std::move(s));
  END_HANDLE_TH_ERRORS
}

// Q, S
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 2);
  const Tensor &q = bytes(a[0], "Q", kCodes, 2), &s = bytes(a[1], "S", kScales, 2);
  const c10::DeviceGuard guard(q.device());
  const int64_t M = q.size(0), K = pair(q, s, "S");
  const std::array<int64_t, 2> sizes{M, K};
  Tensor x = at::empty(sizes, q.options().dtype(at::kBFloat16));
  if (M) {
    const int m = as_int(M, "M"), k = as_int(K, "K");
    void* const stream = stream_on(q);
    call([&] { return dequantize_mxfp4(q.const_data_ptr(), s.const_data_ptr(), x.data_ptr(), m, k, stream); });
  }
  return THPVariable_Wrap(std::move(x));
  END_HANDLE_TH_ERRORS
}

// A, B, a_scale, b_scale, m_indices, out, gated, quantize
PyObject* product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 8);
  const bool grouped = a[4] != Py_None, gated = truth(a[6]), quantized = truth(a[7]);
  const int dim = grouped ? 3 : 2;
  const Tensor &x = bytes(a[0], "A", kCodes, 2), &b = bytes(a[1], "B", kCodes, dim);
  const Tensor &sx = bytes(a[2], "a_scale", kScales, 2), &sb = bytes(a[3], "b_scale", kScales, dim);
  const c10::DeviceGuard guard(x.device());
  on(b, "B", x);
  const int64_t M = x.size(0), K = pair(x, sx, "a_scale");
  TORCH_CHECK_VALUE(pair(b, sb, "b_scale") == K, "A and B disagree on K: ", K, " and ", 2 * b.size(-1));
  const int64_t G = grouped ? b.size(0) : 1, rows = b.size(dim - 2);
  TORCH_CHECK_VALUE(!gated || rows % 2 == 0, "B must hold as many gate rows as up rows, got ", rows, " rows");
  const int64_t N = gated ? rows / 2 : rows;
  const int32_t* ids = grouped ? vector<int32_t>(a[4], "m_indices", M, at::kInt, x) : nullptr;
  TORCH_CHECK_VALUE(!quantized || a[5] == Py_None, "out goes with a BF16 result");
  TORCH_CHECK_VALUE(!quantized || N % 32 == 0, "an MXFP4 result needs a multiple of 32 columns, got ", N);
  Tensor c, s;
  if (quantized) {
    const std::array<int64_t, 2> qs{M, N / 2}, ss{M, N / 32};
    c = empty_bytes(qs, x);
    s = empty_bytes(ss, x);
  } else {
    const std::array<int64_t, 2> sizes{M, N};
    const at::IntArrayRef shape(sizes);
    if (a[5] == Py_None) {
      c = at::empty(shape, x.options().dtype(at::kBFloat16));
    } else {
      c = tensor(a[5], "out", at::kBFloat16, 2);
      TORCH_CHECK_VALUE(c.sizes() == shape && c.device() == x.device() && c.is_contiguous(),
                        "out must be a contiguous bfloat16 tensor of shape ", shape, " on ", x.device());
    }
  }
  if (M) {
    const int m = as_int(M, "M"), nn = as_int(N, "N"), k = as_int(K, "K"), g = as_int(G, "G");
    void* const stream = stream_on(x);
    const void *pa = x.const_data_ptr(), *pb = b.const_data_ptr(), *psa = sx.const_data_ptr(),
               *psb = sb.const_data_ptr();
    void *pc = c.data_ptr(), *ps = quantized ? s.data_ptr() : nullptr;
    call([&] {
      if (gated)
        return grouped ? grouped_mxfp4_gated_gemm(pa, pb, psa, psb, ids, pc, ps, m, nn, k, g, stream)
                       : mxfp4_gated_gemm(pa, pb, psa, psb, pc, ps, m, nn, k, stream);
      return grouped ? grouped_mxfp4_gemm(pa, pb, psa, psb, ids, pc, m, nn, k, g, stream)
                     : mxfp4_gemm(pa, pb, psa, psb, pc, m, nn, k, stream);
    });
  }
  if (quantized) return both(std::move(c), std::move(s));
  return a[5] == Py_None ? THPVariable_Wrap(std::move(c)) : Py_NewRef(a[5]);
  END_HANDLE_TH_ERRORS
}

// x, residual, weight, post_weight, gate, scale, eps, quantize
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 8);
  const Tensor& x = rows_of(a[0], "x");
  const c10::DeviceGuard guard(x.device());
  const int64_t T = x.size(0), H = x.size(1);
  const std::array<int64_t, 2> sizes{T, H};
  const at::IntArrayRef shape(sizes);
  long long strides[3] = {step(x, 0), 0, 0};
  const auto operand = [&](PyObject* o, const char* name, long long& row) -> const void* {
    if (o == Py_None) return nullptr;
    const Tensor& t = rows_of(o, name);
    on(t, name, x);
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " must be ", shape, " as x, got ", t.sizes());
    row = step(t, 0);
    return t.const_data_ptr();
  };
  const void* residual = operand(a[1], "residual", strides[1]);
  const uint16_t* weight = vector<uint16_t>(a[2], "weight", H, at::kBFloat16, x);
  const uint16_t* post = a[3] == Py_None ? nullptr : vector<uint16_t>(a[3], "post_weight", H, at::kBFloat16, x);
  const bool channel = a[4] != Py_None && THPVariable_Check(a[4]) && THPVariable_Unpack(a[4]).dim() == 1;
  const void* gate = channel ? vector<uint16_t>(a[4], "gate", H, at::kBFloat16, x) : operand(a[4], "gate", strides[2]);
  const double scale = PyFloat_AsDouble(a[5]);
  if (scale == -1.0 && PyErr_Occurred()) throw python_error();
  const double eps = PyFloat_AsDouble(a[6]);
  if (eps == -1.0 && PyErr_Occurred()) throw python_error();
  const bool quantized = truth(a[7]);
  TORCH_CHECK_VALUE(!quantized || H % 32 == 0, "an MXFP4 result needs a multiple of 32 columns, got ", H);
  Tensor h = at::empty(shape, x.options()), y, s;
  if (quantized) {
    const std::array<int64_t, 2> qs{T, H / 2}, ss{T, H / 32};
    y = empty_bytes(qs, x);
    s = empty_bytes(ss, x);
  } else {
    y = at::empty(shape, x.options());
  }
  if (T) {
    const int t = as_int(T, "T"), w = as_int(H, "H");
    void* const stream = stream_on(x);
    call([&] {
      return residual_norm(x.const_data_ptr(), residual, gate, strides, post, weight, (float)scale, (float)eps,
                           h.data_ptr(), y.data_ptr(), quantized ? s.data_ptr() : nullptr, t, w, stream);
    });
  }
  THPObjectPtr first(quantized ? both(std::move(y), std::move(s)) : THPVariable_Wrap(std::move(y)));
  if (!first) return nullptr;
  THPObjectPtr second(THPVariable_Wrap(std::move(h)));
  return PyTuple_Pack(2, first.get(), second.get());
  END_HANDLE_TH_ERRORS
}

}  // namespace fgg_binding
