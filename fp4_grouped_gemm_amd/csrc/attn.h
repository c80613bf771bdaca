// Attention operators: the launchers' arguments and the device helpers that
// the three kernels share (the paged cache, types, LDS reads, wave
// reductions).
#pragma once

#include "common.h"

namespace fgg {

// A paged key-value cache: K and V hold num_pages pages of page_size (a
// power of two) tokens of kv_heads heads of D values, BF16 or E4M3 codes
// with one FP32 scale per KV head.  Strides are in bytes, multiples of 16,
// of any order of the page, head and token dimensions; values of a head are
// contiguous.
struct KvCache {
  uint8_t* k;
  uint8_t* v;
  long long k_page, k_head, k_token;
  long long v_page, v_head, v_token;
  const float* k_scale;  // [kv_heads], or nullptr: 1
  const float* v_scale;
  const int32_t* table;  // [batch, width]: the pages of each sequence, in order
  long long table_stride;
  int num_pages, kv_heads, page_shift, batch, width;
  bool fp8;
};

struct AppendArgs {
  KvCache c;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  long long q_token, q_head, k_token, k_head, v_token, v_head;  // strides in values
  const float* turns;  // [npos, rot]: rot / 2 cosines, then rot / 2 sines
  const int32_t* positions;
  const int32_t* seq_ids;  // nullptr: token t belongs to sequence t
  uint16_t* q_out;         // [T, q_heads, D]
  uint16_t* k_out;         // [T, kv_heads, D], or nullptr
  int T, q_heads, D, rot, npos;
  bool interleaved;
};

namespace decode_detail {
// A row that the slices of several workgroups share, for the join; written
// by the workgroup whose slice it begins in.
struct SplitRow {
  int first, last;  // those workgroups; first < 0: no such row
  int b, head0, heads, pad[3];
};
static_assert(sizeof(SplitRow) == 32, "two 16-byte loads");
}  // namespace decode_detail

struct DecodeArgs {
  KvCache c;
  const uint16_t* q;
  long long q_seq, q_head;  // strides in values
  const int32_t* lengths;
  uint16_t* out;  // [batch, q_heads, D]
  float* part_o;  // [workgroups, 2, 16, D] unnormalised outputs of split rows
  float* part_ml; // [workgroups, 2, 16, 2] their maxima (log2 domain) and sums
  decode_detail::SplitRow* split;  // [workgroups] rows to join
  float scale;
  int q_heads, D;
};

struct PromptArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  long long q_token, q_head, k_token, k_head, v_token, v_head;  // strides in values
  const int32_t* starts;  // [batch + 1]
  uint16_t* out;          // [T, q_heads, D]
  float scale;
  int T, batch, q_heads, kv_heads, D;
  int num_cus;  // compute units of the device
};

// Workgroups that share the list of a decode launch, from the longest length
// the table can hold; 0: each row has one of its own.
int decode_workgroups(int batch, int q_heads, int kv_heads, long long max_len, int num_cus);
// Bytes of its workspace (part_o, part_ml, split) for that many workgroups.
size_t decode_workspace(int workgroups, int D);

// Workgroups, of 256 threads, that a prompt launch takes at most.  (Split over the
// keys it takes up to twice as many, but that is done for few workgroups only.)
long long prompt_workgroups(int T, int batch, int q_heads, int kv_heads);

hipError_t launch_append(const AppendArgs& a, hipStream_t s);
hipError_t launch_decode(const DecodeArgs& a, int workgroups, hipStream_t s);
hipError_t launch_prompt(const PromptArgs& a, hipStream_t s);

#ifdef __HIPCC__
namespace attn {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// Two of the four E4M3 codes of a word as two BF16 values (exact: E4M3 has
// three bits of mantissa).
template <bool HIGH>
__device__ __forceinline__ uint32_t fp8x2_to_bf16(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
}
// 8 codes -> 8 BF16 values.
__device__ __forceinline__ u32x4 fp8x8_to_bf16(u32x2 w) {
  return (u32x4){fp8x2_to_bf16<false>(w[0]), fp8x2_to_bf16<true>(w[0]), fp8x2_to_bf16<false>(w[1]),
                 fp8x2_to_bf16<true>(w[1])};
}

// Transposed LDS read: each block of 16 lanes reads 4 rows of 16 16-bit
// values (lane i: values 4 (i % 4) .. + 3 of row i / 4, at its own address)
// and lane i gets the four rows' values of column i.
__device__ __forceinline__ u32x2 lds_read_tr(const uint8_t* p) {
  typedef __attribute__((address_space(3))) s16x4* lds4;
  return __builtin_bit_cast(
      u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(const_cast<uint8_t*>(p))));
}

__device__ __forceinline__ float xor_max(float v, int off) { return fmaxf(v, __shfl_xor(v, off, 64)); }
__device__ __forceinline__ float xor_add(float v, int off) { return v + __shfl_xor(v, off, 64); }

}  // namespace attn
#endif

}  // namespace fgg
