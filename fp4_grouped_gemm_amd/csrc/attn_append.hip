// rope_kv_append: rotates the queries and keys of new tokens by their
// positions and writes keys and values to a paged cache.
//
//   (a, b) -> (a c - b s, b c + a s),  c, s = cos, sin of the position's
// angle for that pair; FP32 (one rounding of each product-sum pair by the
// fused multiply-add), then one rounding to BF16 or to E4M3.
//
// A thread takes 16 values of one head of one token: eight pairs (two
// 16-byte pieces, rot / 2 apart or side by side) or 16 values to copy.  All
// are loads and stores of 16 bytes (8 for codes); nothing is read twice but
// the table, whose rows the heads of a token share in L1/L2.  Bound by HBM, and
// for small calls by the launch: 16665 tokens of 32 + 8 + 8 heads of 128, all
// outputs, 81 us for 452 MB (5.6 TB/s; a copy reaches 5.1), and 80 us for 418 MB with
// an E4M3 cache, whose exact division of each cached value lies under the memory's
// time; one token 3 us on the GPU, 250 tokens of 64 + 8 + 8 heads 5 us.
#include "attn.h"

namespace fgg {
namespace append_detail {

using namespace attn;

constexpr int kThreads = 256;

__device__ __forceinline__ void unpack8(u32x4 w, float v[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ u32x4 to_bf16x8(const float v[8]) {
  return (u32x4){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                 pack_bf16(v[6], v[7])};
}

// E4M3FN_RNE(clamp(x / scale, +-448)); NaN stays NaN.
__device__ __forceinline__ float to_code_range(float x, float scale) {
  const float y = x / scale;
  return y != y ? y : fminf(fmaxf(y, -448.0f), 448.0f);
}
__device__ __forceinline__ u32x2 to_fp8x8(const float v[8], float scale) {
  u32x2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(to_code_range(v[4 * i], scale),
                                            to_code_range(v[4 * i + 1], scale), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(to_code_range(v[4 * i + 2], scale),
                                        to_code_range(v[4 * i + 3], scale), w, true);
    r[i] = (uint32_t)w;
  }
  return r;
}

__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a) {
  const uint32_t pieces = (uint32_t)a.D / 16;  // of a head
  const uint32_t heads = (uint32_t)(a.q_heads + 2 * a.c.kv_heads);
  const uint32_t id = blockIdx.x * kThreads + threadIdx.x;
  const uint32_t row = id / pieces;
  const int u = (int)(id - row * pieces);
  const int t = (int)(row / heads);
  int h = (int)(row - (uint32_t)t * heads);
  if (t >= a.T) return;
  const int pos = a.positions[t];
  const int seq = a.seq_ids ? a.seq_ids[t] : t;
  const bool token = pos >= 0 && pos < a.npos && (pos >> a.c.page_shift) < a.c.width && seq >= 0 &&
                     seq < a.c.batch;
  // which of q, k, v this head belongs to
  const int part = h < a.q_heads ? 0 : h < a.q_heads + a.c.kv_heads ? 1 : 2;
  h -= part == 0 ? 0 : part == 1 ? a.q_heads : a.q_heads + a.c.kv_heads;
  const uint16_t* src = part == 0   ? a.q + (long long)t * a.q_token + h * a.q_head
                        : part == 1 ? a.k + (long long)t * a.k_token + h * a.k_head
                                    : a.v + (long long)t * a.v_token + h * a.v_head;
  const bool turn = part != 2 && u * 16 < a.rot;
  const bool apart = turn && !a.interleaved;  // pairs (i, i + rot / 2)
  const int o0 = apart ? u * 8 : u * 16, o1 = apart ? a.rot / 2 + u * 8 : u * 16 + 8;
  float x[8], y[8];
  if (token) {
    unpack8(*reinterpret_cast<const u32x4*>(src + o0), x);
    unpack8(*reinterpret_cast<const u32x4*>(src + o1), y);
    if (turn) {
      const float* c = a.turns + (long long)pos * a.rot + u * 8;
      const float* s = c + a.rot / 2;
      float cs[8], sn[8];
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<f32x4*>(cs + i) = *reinterpret_cast<const f32x4*>(c + i);
        *reinterpret_cast<f32x4*>(sn + i) = *reinterpret_cast<const f32x4*>(s + i);
      }
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float* z = i < 4 ? x : y;  // pair i is values 2i, 2i + 1 of the 16
          const int j = 2 * (i & 3);
          const float p = z[j], q = z[j + 1];
          z[j] = fmaf(p, cs[i], -q * sn[i]);
          z[j + 1] = fmaf(q, cs[i], p * sn[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = x[i], q = y[i];
          x[i] = fmaf(p, cs[i], -q * sn[i]);
          y[i] = fmaf(q, cs[i], p * sn[i]);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
  }
  uint16_t* plain = part == 0   ? a.q_out + ((long long)t * a.q_heads + h) * a.D
                    : part == 1 && a.k_out ? a.k_out + ((long long)t * a.c.kv_heads + h) * a.D
                                           : nullptr;
  if (plain) {
    *reinterpret_cast<u32x4*>(plain + o0) = to_bf16x8(x);
    *reinterpret_cast<u32x4*>(plain + o1) = to_bf16x8(y);
  }
  if (part == 0 || !token) return;
  const int page = a.c.table[(long long)seq * a.c.table_stride + (pos >> a.c.page_shift)];
  if (page < 0 || page >= a.c.num_pages) return;
  const int slot = pos & ((1 << a.c.page_shift) - 1);
  uint8_t* dst = part == 1 ? a.c.k + page * a.c.k_page + h * a.c.k_head + slot * a.c.k_token
                           : a.c.v + page * a.c.v_page + h * a.c.v_head + slot * a.c.v_token;
  if (a.c.fp8) {
    const float* sc = part == 1 ? a.c.k_scale : a.c.v_scale;
    const float scale = sc ? sc[h] : 1.0f;
    *reinterpret_cast<u32x2*>(dst + o0) = to_fp8x8(x, scale);
    *reinterpret_cast<u32x2*>(dst + o1) = to_fp8x8(y, scale);
  } else {
    *reinterpret_cast<u32x4*>(dst + 2 * o0) = to_bf16x8(x);
    *reinterpret_cast<u32x4*>(dst + 2 * o1) = to_bf16x8(y);
  }
}

}  // namespace append_detail

hipError_t launch_append(const AppendArgs& a, hipStream_t s) {
  using namespace append_detail;
  const long long n = (long long)a.T * (a.q_heads + 2 * a.c.kv_heads) * (a.D / 16);
  if (n <= 0) return hipSuccess;
  if (n > 0x7FFFFFFFLL) return hipErrorInvalidValue;  // indexes of 32 bits (the host checks)
  hipLaunchKernelGGL(append_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads),
                     0, s, a);
  return hipGetLastError();
}

}  // namespace fgg
