// MXFP4 (E2M1 codes, one power of two per 32 of them along a row) and the norm
// at a block's border: the launchers' arguments and the device helpers that
// their kernels share.
//
// A block's scale is an E8M0 code e, the value 2^(e - 127); 255 is NaN.  Of a
// block whose largest magnitude lies in [2^p, 2^(p + 1)) it is e = max(p - 2 +
// 127, 0), so that this magnitude over the scale lies in [4, 8); codes are
// rounded to nearest, ties to even, and saturate at 6.  A block that holds an
// infinity or a NaN gets e = 255 and codes of zero: what it reaches is NaN.
#pragma once

#include "common.h"

namespace fgg {

// Products of A [M, K] with B, MXFP4 both: B [G, N, K], or for gated ones
// [G, 2 N, K], the N gate rows before the N up rows.
struct MxGemmArgs {
  const uint8_t* A;        // [M, K / 2]
  const uint8_t* B;        // [G, N or 2 N, K / 2]
  const uint8_t* a_scale;  // [M, K / 32]
  const uint8_t* b_scale;  // [G, N or 2 N, K / 32]
  const int32_t* m_indices;  // nullptr: every row is expert 0
  uint8_t* C;              // [M, N] BF16, or [M, N / 2] codes
  uint8_t* c_scale;        // [M, N / 32], or nullptr: BF16
  int M, N, K, G;
  bool gated;
  int num_cus;
};

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;     // or nullptr: 0
  const uint16_t* gate;         // or nullptr: 1
  const uint16_t* post_weight;  // or nullptr: x is not normed
  const uint16_t* weight;
  long long x_row, residual_row, gate_row;  // strides in values
  uint16_t* h;       // [T, H]
  uint8_t* y;        // [T, H] BF16, or [T, H / 2] codes
  uint8_t* y_scale;  // [T, H / 32], or nullptr: BF16
  float scale, eps;
  int T, H;
};

hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t s);
hipError_t launch_mx_rows(const MxGemmArgs& a, hipStream_t s);                // few rows: a stream of the weights
hipError_t launch_mx_tiles(const MxGemmArgs& a, bool large, hipStream_t s);  // many rows
hipError_t launch_norm(const NormArgs& a, hipStream_t s);
// rows as for the other quantisers
hipError_t launch_quant_mxfp4(const uint16_t* X, uint8_t* Q, uint8_t* S, int M, int K, int num_cus,
                              hipStream_t s, const int32_t* rows = nullptr, int T = 0);
hipError_t launch_dequant_mxfp4(const uint8_t* Q, const uint8_t* S, uint16_t* X, int M, int K,
                                int num_cus, hipStream_t s);

#ifdef __HIPCC__
namespace mx {

// E8M0 code of a block whose largest magnitude has the FP32 bits `top`.
__device__ __forceinline__ uint32_t scale_code(uint32_t top) {
  const int e = (int)(top >> 23);
  return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}
// 1 / 2^(code - 127), a normal FP32 for the codes that scale_code gives;
// 0 for 255.
__device__ __forceinline__ float inverse(uint32_t code) {
  return code == 255u ? 0.0f : __uint_as_float((254u - code) << 23);
}
// 2^(code - 127), NaN for 255.
__device__ __forceinline__ float value(uint32_t code) {
  return __uint_as_float(code == 0u ? 0x00400000u : code == 255u ? 0x7FC00000u : code << 23);
}

// 8 values times inv (a power of two: exact but for values far below half a
// code) -> 8 E2M1 codes, value 2 j in the low half of byte j.  The convert
// rounds to nearest even; its operands are within +-6, so that its own
// treatment of larger ones does not matter.
__device__ __forceinline__ uint32_t codes8(const float v[8], float inv) {
  uint32_t packed = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float a = fminf(fmaxf(v[i] * inv, -6.0f), 6.0f);
    const float b = fminf(fmaxf(v[i + 1] * inv, -6.0f), 6.0f);
    packed |= ((uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, a, b, 1.0f, 0) & 0xFFu) << (4 * i);
  }
  return packed;
}

// Largest magnitude of 8 values as FP32 bits: ordered like the magnitudes,
// infinities and NaN above all numbers.
__device__ __forceinline__ uint32_t top8(const float v[8]) {
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return t;
}

// silu(gate) * up in FP32: gate / (1 + exp(-gate)) is -0 where the
// exponential overflows.
__device__ __forceinline__ float gated(float gate, float up) {
  return gate / (1.0f + expf(-gate)) * up;
}

}  // namespace mx
#endif

}  // namespace fgg
