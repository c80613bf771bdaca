// The attention operators' binding: checks tensors, allocates results, and calls
// the C ABI (include/fgg.h).  Compiled because the calls are short: one token's
// append takes 3 us on the GPU and its launch 3.7 us of the host, and the same
// checks and argument conversions written in Python took another 5.5.
//
// The functions take attention.py's arguments by position, run on the current
// stream of their operands' device, and raise ValueError for everything that they
// or the library refuse.
#include <array>
#include <cmath>

#include "binding.h"

namespace {

using namespace fgg_binding;

// A BF16 [rows, heads, head_dim] operand, head_dim contiguous.
const Tensor& heads(PyObject* o, const char* name) {
  const Tensor& t = tensor(o, name, at::kBFloat16, 3);
  TORCH_CHECK_VALUE(t.stride(2) == 1, name, " must be contiguous in its last dimension");
  return t;
}

// A 2-D tensor on q's device, its last dimension contiguous.
const Tensor& matrix(PyObject* o, const char* name, at::ScalarType dtype, const Tensor& q) {
  const Tensor& t = tensor(o, name, dtype, 2);
  on(t, name, q);
  TORCH_CHECK_VALUE(t.stride(1) == 1 || t.size(1) == 1, name, " must be contiguous in its last dimension");
  return t;
}

const Tensor& pool(PyObject* o, const char* name, const Tensor& q) {
  TORCH_CHECK_VALUE(THPVariable_Check(o) && THPVariable_Unpack(o).dim() == 4, name,
                    " must be a tensor [pages, kv_heads, page_size, head_dim]");
  const Tensor& t = THPVariable_Unpack(o);
  TORCH_CHECK_VALUE(t.device() == q.device(), name, " is on ", t.device(), ", expected ", q.device());
  TORCH_CHECK_VALUE(t.stride(3) == 1, "k_cache and v_cache must be contiguous in their last dimension");
  return t;
}

fgg_kv_cache cache(PyObject* k_, PyObject* v_, PyObject* table_, PyObject* k_scale, PyObject* v_scale,
                   const Tensor& q) {
  const Tensor &k = pool(k_, "k_cache", q), &v = pool(v_, "v_cache", q);
  TORCH_CHECK_VALUE(k.scalar_type() == v.scalar_type() && k.sizes() == v.sizes(),
                    "k_cache and v_cache must have one dtype and shape");
  const bool fp8 = k.scalar_type() == at::kFloat8_e4m3fn || k.scalar_type() == at::kByte;
  TORCH_CHECK_VALUE(fp8 || k.scalar_type() == at::kBFloat16,
                    "a cache holds bfloat16 or E4M3 codes (float8_e4m3fn / uint8), got ",
                    type_name(k.scalar_type()));
  const Tensor& table = matrix(table_, "page_table", at::kInt, q);
  TORCH_CHECK_VALUE(fp8 || (k_scale == Py_None && v_scale == Py_None),
                    "k_scale and v_scale go with an E4M3 cache");
  for (const Tensor* t : {&k, &table})
    for (int64_t n : t->sizes()) TORCH_CHECK_VALUE(n <= INT32_MAX, "a cache dimension passes 2^31");
  fgg_kv_cache c{};
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.k_scale = k_scale == Py_None ? nullptr : vector<float>(k_scale, "k_scale", k.size(1), at::kFloat, q);
  c.v_scale = v_scale == Py_None ? nullptr : vector<float>(v_scale, "v_scale", k.size(1), at::kFloat, q);
  c.page_table = static_cast<const int32_t*>(table.const_data_ptr());
  c.table_stride = step(table, 0);
  for (int i = 0; i < 3; ++i) {
    c.k_strides[i] = step(k, i);
    c.v_strides[i] = step(v, i);
  }
  c.dtype = fp8 ? FGG_KV_E4M3 : FGG_KV_BF16;
  c.num_pages = (int)k.size(0);
  c.kv_heads = (int)k.size(1);
  c.page_size = (int)k.size(2);
  c.head_dim = (int)k.size(3);
  c.batch = (int)table.size(0);
  c.table_width = (int)table.size(1);
  return c;
}

// `out` if given, else a new BF16 tensor [rows, heads, dim] like q.
Tensor result(PyObject* out, const Tensor& q, int64_t rows, int64_t n, int64_t dim) {
  if (out == Py_None) return at::empty({rows, n, dim}, q.options());
  const std::array<int64_t, 3> sizes{rows, n, dim};
  const at::IntArrayRef shape(sizes);
  TORCH_CHECK_VALUE(THPVariable_Check(out), "out must be a tensor");
  const Tensor& t = THPVariable_Unpack(out);
  TORCH_CHECK_VALUE(t.scalar_type() == at::kBFloat16 && t.sizes() == shape && t.device() == q.device() &&
                        t.is_contiguous(),
                    "out must be a contiguous bfloat16 tensor of shape ", shape, " on ", q.device());
  return t;
}

float scale_of(PyObject* o, int64_t dim) {
  if (o == Py_None) return 1.0f / std::sqrt((float)dim);
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)x;
}

// q, k, v, cos_sin, positions, page_table, k_cache, v_cache, seq_ids, interleaved,
// k_scale, v_scale, return_k, out
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 14);
  const Tensor &q = heads(a[0], "q"), &k = heads(a[1], "k"), &v = heads(a[2], "v");
  on(k, "k", q);
  on(v, "v", q);
  const c10::DeviceGuard guard(q.device());
  const fgg_kv_cache c = cache(a[6], a[7], a[5], a[10], a[11], q);
  const int64_t T = q.size(0), hq = q.size(1), d = q.size(2), hk = c.kv_heads;
  const std::array<int64_t, 3> kv_sizes{T, hk, d};
  const at::IntArrayRef kv(kv_sizes);
  TORCH_CHECK_VALUE(d == c.head_dim && k.sizes() == kv && v.sizes() == kv, "q must be [T, Hq, ", c.head_dim,
                    "], k and v [T, ", hk, ", ", c.head_dim, "] as the cache");
  const Tensor& turns = matrix(a[3], "cos_sin", at::kFloat, q);
  TORCH_CHECK_VALUE(turns.stride(0) == turns.size(1) || turns.size(0) == 1, "cos_sin must be contiguous");
  const int32_t* pos = vector<int32_t>(a[4], "positions", T, at::kInt, q);
  const int32_t* ids = a[8] == Py_None ? nullptr : vector<int32_t>(a[8], "seq_ids", T, at::kInt, q);
  const bool return_k = truth(a[12]);
  Tensor res = result(a[13], q, T, hq, d), k_out;
  if (return_k) k_out = at::empty({T, hk, d}, q.options());
  if (T) {
    const long long strides[6] = {step(q, 0), step(q, 1), step(k, 0), step(k, 1), step(v, 0), step(v, 1)};
    const int num = as_int(turns.size(0), "cos_sin"), rot = as_int(turns.size(1), "cos_sin");
    const int tokens = as_int(T, "T"), q_heads = as_int(hq, "Hq"), interleaved = truth(a[9]);
    void* const stream = stream_on(q);
    call([&] {
      return rope_kv_append(&c, q.const_data_ptr(), k.const_data_ptr(), v.const_data_ptr(), strides,
                            static_cast<const float*>(turns.const_data_ptr()), num, rot, interleaved, pos, ids,
                            res.data_ptr(), return_k ? k_out.data_ptr() : nullptr, tokens, q_heads, stream);
    });
  }
  THPObjectPtr first(a[13] == Py_None ? THPVariable_Wrap(std::move(res)) : Py_NewRef(a[13]));
  if (!return_k) return first.release();
  THPObjectPtr second(THPVariable_Wrap(std::move(k_out)));
  return PyTuple_Pack(2, first.get(), second.get());
  END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, page_table, lengths, scale, k_scale, v_scale, out
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 9);
  const Tensor& q = heads(a[0], "q");
  const c10::DeviceGuard guard(q.device());
  const fgg_kv_cache c = cache(a[1], a[2], a[3], a[6], a[7], q);
  const int64_t B = q.size(0), hq = q.size(1), d = q.size(2);
  TORCH_CHECK_VALUE(d == c.head_dim && B == c.batch, "q must be [", c.batch, ", Hq, ", c.head_dim,
                    "] as the page table and the cache");
  const int32_t* lens = vector<int32_t>(a[4], "lengths", B, at::kInt, q);
  const float scale = scale_of(a[5], d);
  Tensor res = result(a[8], q, B, hq, d);
  if (B) {
    size_t need = 0;
    const int q_heads = as_int(hq, "Hq");
    call([&] { return paged_decode_attention_workspace(&c, q_heads, &need); });
    // (a call that needs no workspace is given its output's address)
    const Tensor work = need ? at::empty({(int64_t)need}, q.options().dtype(at::kByte)) : res;
    void* const stream = stream_on(q);
    call([&] {
      return paged_decode_attention(&c, q.const_data_ptr(), step(q, 0), step(q, 1), lens, scale, res.data_ptr(),
                                    q_heads, work.data_ptr(), need, stream);
    });
  }
  return a[8] == Py_None ? THPVariable_Wrap(std::move(res)) : Py_NewRef(a[8]);
  END_HANDLE_TH_ERRORS
}

// q, k, v, starts, scale, out
PyObject* prompt(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 6);
  const Tensor &q = heads(a[0], "q"), &k = heads(a[1], "k"), &v = heads(a[2], "v");
  on(k, "k", q);
  on(v, "v", q);
  const c10::DeviceGuard guard(q.device());
  const int64_t T = q.size(0), hq = q.size(1), d = q.size(2), hk = k.size(1);
  const std::array<int64_t, 3> kv_sizes{T, hk, d};
  const at::IntArrayRef kv(kv_sizes);
  TORCH_CHECK_VALUE(k.sizes() == kv && v.sizes() == kv, "k and v must be [", T, ", Hkv, ", d, "] as q");
  const int32_t* starts = vector<int32_t>(a[3], "starts", -1, at::kInt, q);
  const int64_t batch = THPVariable_Unpack(a[3]).size(0) - 1;
  TORCH_CHECK_VALUE(batch >= 1, "starts must be an int32 tensor of shape (B + 1,), B >= 1");
  const float scale = scale_of(a[4], d);
  Tensor res = result(a[5], q, T, hq, d);
  if (T) {
    const long long strides[6] = {step(q, 0), step(q, 1), step(k, 0), step(k, 1), step(v, 0), step(v, 1)};
    const int tokens = as_int(T, "T"), prompts = as_int(batch, "B"), q_heads = as_int(hq, "Hq"),
              kv_heads = as_int(hk, "Hkv"), dim = as_int(d, "D");
    void* const stream = stream_on(q);
    call([&] {
      return prompt_attention(q.const_data_ptr(), k.const_data_ptr(), v.const_data_ptr(), strides, starts, scale,
                              res.data_ptr(), tokens, prompts, q_heads, kv_heads, dim, stream);
    });
  }
  return a[5] == Py_None ? THPVariable_Wrap(std::move(res)) : Py_NewRef(a[5]);
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {method<append>("rope_kv_append"), method<decode>("paged_decode_attention"),
                         method<prompt>("prompt_attention"), method<quantize>("quantize_mxfp4"),
                         method<dequantize>("dequantize_mxfp4"), method<product>("mxfp4_product"),
                         method<norm>("residual_norm"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attention", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attention() { return PyModule_Create(&module); }
