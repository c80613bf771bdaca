// The border between two blocks of a layer in one pass: the sum of a block's
// output into the residual, and the norm that the next block reads.
//
//   u = x, or post_weight * x / sqrt(mean(x^2) + eps)
//   h = residual + scale * gate * u                        (written as BF16)
//   y = weight * h / sqrt(mean(h^2) + eps)                 (BF16 or MXFP4)
//
// All in FP32, the means over a row of H values included; y is taken from the
// FP32 h, not from its rounded copy.  Bound by memory: x, residual (and a gate
// of its own for each token) are read once, h and y written once; a row's
// values stay in the registers of the one or four waves that hold it, eight
// consecutive ones (16 bytes) a lane.  Rows of more values than those
// registers take are read three times.
//
// Measured: 8192 rows of 7168, both norms and a gate for each channel, 470 MB, 101
// us (4.6 TB/s, what a copy on this card reaches); one row of 4096 4.8 us where
// launches follow each other, 3.0 on the GPU.
#include "mx.h"

namespace fgg {
namespace norm_detail {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void load8(const uint16_t* p, float v[8]) {
  const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store8(uint16_t* p, const float v[8]) {
  const uint2 lo = pack_bf16x4(v[0], v[1], v[2], v[3]), hi = pack_bf16x4(v[4], v[5], v[6], v[7]);
  *reinterpret_cast<uint4*>(p) = make_uint4(lo.x, lo.y, hi.x, hi.y);
}

// Sum over a row's W waves, in a fixed order: every thread gets the same value.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off, 64);
  if constexpr (W > 1) {
    __syncthreads();  // the last sum's readers are done
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += red[w];
  }
  return v;
}

__device__ __forceinline__ float squares(const float v[8], float sum) {
#pragma unroll
  for (int i = 0; i < 8; ++i) sum = fmaf(v[i], v[i], sum);
  return sum;
}

// u -> h of the eight values at column c
__device__ __forceinline__ void residual8(const NormArgs& a, long long row, int c, bool post, float rs,
                                          float v[8]) {
  float w[8];
  if (post) {
    load8(a.post_weight + c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * rs * w[i];
  }
  if (a.gate) {
    load8(a.gate + row * a.gate_row + c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= w[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 0.f;
  if (a.residual) load8(a.residual + row * a.residual_row + c, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = fmaf(a.scale, v[i], w[i]);
}

// h and y of the eight values at column c; four lanes hold a block of 32.
__device__ __forceinline__ void finish8(const NormArgs& a, long long row, int c, float rs, const float v[8]) {
  store8(a.h + row * a.H + c, v);
  float w[8];
  load8(a.weight + c, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = v[i] * rs * w[i];
  if (a.y_scale) {
    uint32_t top = mx::top8(w);
    top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
    const uint32_t code = mx::scale_code(top);
    *reinterpret_cast<uint32_t*>(a.y + (row * a.H + c) / 2) =
        code == 255u ? 0u : mx::codes8(w, mx::inverse(code));
    if (c % 32 == 0) a.y_scale[(row * a.H + c) / 32] = (uint8_t)code;
  } else {
    store8(reinterpret_cast<uint16_t*>(a.y) + row * a.H + c, w);
  }
}

__device__ __forceinline__ float inverse_rms(float sum, const NormArgs& a) {
  return 1.0f / sqrtf(sum / (float)a.H + a.eps);
}

// W waves a row (1: a row a wave, 4: a row a workgroup), at most U pieces of
// eight values a lane.
template <int W, int U>
__global__ __launch_bounds__(256) void norm_kernel(const NormArgs a) {
  __shared__ float red[4];
  const long long row = W == 1 ? (long long)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (W == 1 && row >= a.T) return;  // (no barrier follows)
  const int t = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  float v[U][8];
  float sum = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (u * 64 * W + t) * 8;
    if (c < a.H) {
      load8(a.x + row * a.x_row + c, v[u]);
      sum = squares(v[u], sum);
    }
  }
  float rs = 1.f;
  const bool post = a.post_weight != nullptr;
  if (post) rs = inverse_rms(row_sum<W>(sum, red), a);
  sum = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (u * 64 * W + t) * 8;
    if (c < a.H) {
      residual8(a, row, c, post, rs, v[u]);
      sum = squares(v[u], sum);
    }
  }
  rs = inverse_rms(row_sum<W>(sum, red), a);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (u * 64 * W + t) * 8;
    if (c < a.H) finish8(a, row, c, rs, v[u]);
  }
}

// Eight sums of squares, each of one place of a lane's pieces: at most H / 2048
// roundings follow each other where one sum of all has H / 256.  A row of 2^20 values
// whose first ones are large loses 2e-4 of a single sum, 3e-5 of these.
struct Sums {
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(const float v[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = fmaf(v[i], v[i], s[i]);
  }
  __device__ __forceinline__ float all() const {
    return ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  }
};

// Rows of any length.
__global__ __launch_bounds__(256) void norm_long_kernel(const NormArgs a) {
  __shared__ float red[4];
  const long long row = blockIdx.x;
  const bool post = a.post_weight != nullptr;
  float v[8], rs = 1.f;
  if (post) {
    Sums sum;
    for (int c = threadIdx.x * 8; c < a.H; c += 2048) {
      load8(a.x + row * a.x_row + c, v);
      sum.add(v);
    }
    rs = inverse_rms(row_sum<4>(sum.all(), red), a);
  }
  Sums sum;
  for (int c = threadIdx.x * 8; c < a.H; c += 2048) {
    load8(a.x + row * a.x_row + c, v);
    residual8(a, row, c, post, rs, v);
    sum.add(v);
  }
  const float rh = inverse_rms(row_sum<4>(sum.all(), red), a);
  for (int c = threadIdx.x * 8; c < a.H; c += 2048) {
    load8(a.x + row * a.x_row + c, v);
    residual8(a, row, c, post, rs, v);
    finish8(a, row, c, rh, v);
  }
}

template <int W, int U>
hipError_t launch(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((norm_kernel<W, U>), dim3((unsigned)(W == 1 ? (a.T + 3) / 4 : a.T)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace norm_detail

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  using namespace norm_detail;
  if (a.H <= 512) return launch<1, 1>(a, s);
  if (a.H <= 1024) return launch<1, 2>(a, s);
  if (a.H <= 2048) return launch<4, 1>(a, s);
  if (a.H <= 4096) return launch<4, 2>(a, s);
  if (a.H <= 8192) return launch<4, 4>(a, s);
  if (a.H <= 16384) return launch<4, 8>(a, s);
  hipLaunchKernelGGL(norm_long_kernel, dim3((unsigned)a.T), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace fgg
