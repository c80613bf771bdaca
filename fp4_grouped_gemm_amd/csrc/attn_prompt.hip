// prompt_attention: causal attention over whole prompts packed one after the
// other, grouped query heads.
//
//   o[t, h] = sum_{u <= t} p_u v_u / sum_{u <= t} p_u,
//   p_u = exp(scale q[t, h] . k[u] - m),  m = max_{u <= t} scale q[t, h] . k[u]
//
// over the tokens u of t's prompt.  A workgroup takes 128 queries of one
// head, 32 a wave, and goes once over the keys in tiles of 64 with the
// running maximum and sum.  S^T = K Q^T on 32x32x16 MFMAs leaves a query's
// scores in one column of two lanes (l and l + 32), so the softmax needs one
// exchange a tile; packed to BF16 the scores are the B operand of
// O^T = V^T P^T as they stand (contraction slot 8 h + 4 a + i of step s is
// token 16 s + 8 a + 4 h + i), with V^T read from LDS by transposed reads.
// Bound by the matrix cores: 4 D operations a query and key.  P is rounded
// to BF16, the matrix cores' input type; scores, maxima, sums and outputs
// are FP32.
//
// A masked value must not reach the output even where it is infinite or NaN:
// masked scores are overwritten, but in the product with V a weight of 0
// times such a value is NaN.  Only the tiles on the diagonal hold values that
// some queries of the workgroup see and others do not; those are looked over
// as they are staged, and in the rare tile that holds a value that is not
// finite, such values are staged as zeros for the product and added by hand
// to the queries that see them.
#include "attn.h"

namespace fgg {
namespace prompt_detail {

using namespace attn;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kRows = 32 * kWaves;  // queries of a workgroup
constexpr int kKeys = 64;           // keys of a tile

// Segment i of the packed tokens: 0 is what lies before the first prompt,
// 1 .. batch the prompts, batch + 1 what lies after the last.  Every bound is
// clamped to [0, T], and a segment that would end before it starts is empty.
__device__ __forceinline__ void segment(const PromptArgs& a, int i, int& lo, int& hi) {
  lo = i == 0 ? 0 : min(max(a.starts[i - 1], 0), a.T);
  hi = i > a.batch ? a.T : min(max(a.starts[i], 0), a.T);
  if (hi < lo) hi = lo;
}
__device__ __forceinline__ int row_tiles(int lo, int hi) { return (hi - lo + kRows - 1) / kRows; }

// Whether one of eight BF16 values is infinite or NaN.
__device__ __forceinline__ bool any_odd(u32x4 w) {
  bool odd = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    odd |= (w[i] & 0x7F80u) == 0x7F80u || (w[i] & 0x7F800000u) == 0x7F800000u;
  return odd;
}

template <int D>
__global__ __launch_bounds__(kThreads, 2) void prompt_kernel(PromptArgs a) {
  constexpr int kSteps = D / 16;   // k-steps of a QK product
  constexpr int kBlocks = D / 32;  // 32-row blocks of O^T
  constexpr int kKRow = D * 2 + 16, kVRow = D * 2 + 32;  // LDS bytes of a staged row
  constexpr int kLanesPerRow = D / 8;
  constexpr int kLoads = kKeys * kLanesPerRow / kThreads;  // 16-byte pieces of a tile per thread
  __shared__ __align__(16) uint8_t ks[kKeys * kKRow];
  __shared__ __align__(16) uint8_t vs[kKeys * kVRow];
  __shared__ int scan_lds[kWaves];
  __shared__ int my_seg, my_tile;
  __shared__ int odd_tile;  // first key + 1 of the last tile with a value that is not finite

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;

  // the row tile of this workgroup: heads fastest, so that the workgroups of
  // one KV head meet on the same XCDs' L2
  const int hid = (int)blockIdx.x % a.q_heads, item = (int)blockIdx.x / a.q_heads;
  const int kvh = hid % a.kv_heads;
  const int head = kvh * (a.q_heads / a.kv_heads) + hid / a.kv_heads;
  {
    const int segs = a.batch + 2, per = (segs + kThreads - 1) / kThreads;
    const int i0 = tid * per, i1 = min(i0 + per, segs);
    int sum = 0, lo, hi, base;
    for (int i = i0; i < i1; ++i) {
      segment(a, i, lo, hi);
      sum += row_tiles(lo, hi);
    }
    if (tid == 0) {
      my_seg = -1;
      odd_tile = 0;
    }
    block_scan<kThreads>(sum, base, scan_lds);
    for (int i = i0; i < i1; ++i) {
      segment(a, i, lo, hi);
      const int n = row_tiles(lo, hi);
      if (base <= item && item < base + n) {
        my_seg = i;
        my_tile = n - 1 - (item - base);  // the tiles with the most keys first
      }
      base += n;
    }
  }
  __syncthreads();
  const int seg = __builtin_amdgcn_readfirstlane(my_seg);
  if (seg < 0) return;
  int lo, hi;
  segment(a, seg, lo, hi);
  const int len = hi - lo;
  const int r0 = __builtin_amdgcn_readfirstlane(my_tile) * kRows;
  const int w0 = r0 + wave * 32;  // this wave's first query
  const int query = w0 + col;
  const bool real = seg >= 1 && seg <= a.batch;

  f32x16 acc[kBlocks];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[i][j] = 0.f;
  float m = kNegInf, l = 0.f;

  if (real) {
    const float scale2 = a.scale * kLog2e;
    bf16x8 qf[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      u32x4 w = {0, 0, 0, 0};
      if (query < len)
        w = *reinterpret_cast<const u32x4*>(a.q + (long long)(lo + query) * a.q_token +
                                            head * a.q_head + s * 16 + half * 8);
      qf[s] = __builtin_bit_cast(bf16x8, w);
    }
    const uint16_t* kp = a.k + (long long)lo * a.k_token + kvh * a.k_head;
    const uint16_t* vp = a.v + (long long)lo * a.v_token + kvh * a.v_head;
    const int keys = min(len, r0 + kRows);  // that any query of the workgroup sees
    u32x4 kw[kLoads], vw[kLoads];
    auto load = [&](int k0) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = k0 + i * (kThreads / kLanesPerRow) + tid / kLanesPerRow;
        const int c = (tid % kLanesPerRow) * 8;
        kw[i] = vw[i] = (u32x4){0, 0, 0, 0};
        if (r < keys) {
          kw[i] = *reinterpret_cast<const u32x4*>(kp + (long long)r * a.k_token + c);
          vw[i] = *reinterpret_cast<const u32x4*>(vp + (long long)r * a.v_token + c);
        }
      }
    };
    load(0);
    for (int k0 = 0; k0 < keys; k0 += kKeys) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = i * (kThreads / kLanesPerRow) + tid / kLanesPerRow;
        const int c = (tid % kLanesPerRow) * 16;
        *reinterpret_cast<u32x4*>(ks + r * kKRow + c) = kw[i];
        *reinterpret_cast<u32x4*>(vs + r * kVRow + c) = vw[i];
      }
      const bool diagonal = k0 + kKeys - 1 > r0;
      if (diagonal) {
        bool odd = false;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) odd |= any_odd(vw[i]);
        if (odd) odd_tile = k0 + 1;
      }
      __syncthreads();
      const bool odd = diagonal && odd_tile == k0 + 1;
      if (odd) {
        for (int x = tid; x < kKeys * D; x += kThreads) {
          uint16_t* w = reinterpret_cast<uint16_t*>(vs + (x / D) * kVRow) + x % D;
          if ((*w & 0x7F80u) == 0x7F80u) *w = 0;
        }
        __syncthreads();
      }
      if (k0 + kKeys < keys) load(k0 + kKeys);
      if (k0 > w0 + 31) continue;  // every key lies after every query of the wave
      f32x16 s[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int j = 0; j < 16; ++j) s[b][j] = 0.f;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const bf16x8 kf = *reinterpret_cast<const bf16x8*>(ks + (b * 32 + col) * kKRow + k * 32 +
                                                             half * 16);
          s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[k], s[b], 0, 0, 0);
        }
      }
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int j = 0; j < 16; ++j) s[b][j] *= scale2;
      if (k0 + kKeys - 1 > w0) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (k0 + b * 32 + (j & 3) + 8 * (j >> 2) + 4 * half > query) s[b][j] = kNegInf;
      }
      float mx = kNegInf;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int j = 0; j < 16; ++j) mx = fmaxf(mx, s[b][j]);
      mx = xor_max(mx, 32);
      const float m1 = fmaxf(m, mx);
      const float ms = m1 == kNegInf ? 0.f : m1;
      const float alpha = __builtin_amdgcn_exp2f(m - ms);
      m = m1;
      float sum = 0.f;
      bf16x8 pf[2][2];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float p[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            p[j] = __builtin_amdgcn_exp2f(s[b][k * 8 + j] - ms);
            sum += p[j];
          }
          pf[b][k] = __builtin_bit_cast(
              bf16x8, (u32x4){pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]),
                              pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7])});
        }
      l = l * alpha + sum;
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) {
        acc[i] *= alpha;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint8_t* src = vs + (b * 32 + k * 16 + half * 4 + ((lane & 15) >> 2)) * kVRow +
                                 i * 64 + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
            const u32x2 x = lds_read_tr(src), y = lds_read_tr(src + 8 * kVRow);
            const bf16x8 vf = __builtin_bit_cast(bf16x8, (u32x4){x[0], x[1], y[0], y[1]});
            acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[b][k], acc[i], 0, 0, 0);
          }
      }
      if (odd && query < len) {
        for (int u = k0; u <= min(query, k0 + kKeys - 1); ++u) {
          const uint16_t* v = vp + (long long)u * a.v_token;
#pragma unroll
          for (int i = 0; i < kBlocks; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const uint32_t w = v[i * 32 + (j & 3) + 8 * (j >> 2) + 4 * half];
              if ((w & 0x7F80u) == 0x7F80u) acc[i][j] += __uint_as_float(w << 16);
            }
        }
      }
    }
    l = xor_add(l, 32);
  }
  if (query >= len) return;
  const float r = l == 0.f ? 0.f : 1.0f / l;
  uint16_t* out = a.out + ((long long)(lo + query) * a.q_heads + head) * D;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<uint2*>(out + i * 32 + j * 8 + half * 4) =
          pack_bf16x4(acc[i][j * 4] * r, acc[i][j * 4 + 1] * r, acc[i][j * 4 + 2] * r,
                      acc[i][j * 4 + 3] * r);
}

}  // namespace prompt_detail

using namespace prompt_detail;

hipError_t launch_prompt(const PromptArgs& a, hipStream_t s) {
  // at most one partly filled tile a segment
  const long long tiles = (long long)a.T / kRows + a.batch + 2;
  const long long grid = tiles * a.q_heads;
  if (grid > 0x7FFFFFFFLL) return hipErrorInvalidValue;  // the host checks
  if (a.D == 64)
    hipLaunchKernelGGL((prompt_kernel<64>), dim3((unsigned)grid), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((prompt_kernel<128>), dim3((unsigned)grid), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace fgg
