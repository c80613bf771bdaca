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

#include <type_traits>

namespace fgg {
namespace prompt_detail {

using namespace attn;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kRows = 32 * kWaves;  // queries of a workgroup
constexpr int kKeys = 64;           // keys of a tile
constexpr float kSlack = 8.f;       // weights may reach 2^kSlack before a rescaling

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

// LDS layout of a staged tile: row r at r D 2 bytes, its 16-byte chunk c at
// chunk c ^ key(r), so that what one cycle of a fragment read touches lies in
// different banks.  K: 16 lanes read one chunk index of 16 rows that differ in
// their low four bits.  V (transposed reads): groups of lanes read 64 bytes
// of four consecutive rows, or 32 bytes of eight.
template <int D>
__device__ __forceinline__ int k_key(int r) {
  return D == 128 ? r & 15 : (r >> 1) & 7;
}
template <int D>
__device__ __forceinline__ int v_key(int r) {
  return D == 128 ? ((r & 3) << 2) | ((r >> 1) & 2) : ((r << 1) & 4) | ((r >> 1) & 2);
}

// Maximum over a lane and its partner in the other half of the wave.
__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

template <int D>
__global__ __launch_bounds__(kThreads, 2) void prompt_kernel(PromptArgs a) {
  constexpr int kSteps = D / 16;    // k-steps of a QK product
  constexpr int kBlocks = D / 32;   // 32-row blocks of O^T
  constexpr int kRowBytes = D * 2;
  constexpr int kBlockBytes = 32 * kRowBytes;  // of a block of 32 keys
  constexpr int kChunks = D / 8;    // 16-byte chunks of a row
  constexpr int kLoads = kBlockBytes / 16 / kThreads;  // chunks of a block per thread
  // rings of four blocks of K and four of V: two are read while two land
  __shared__ __align__(16) uint8_t lds[8 * kBlockBytes];
  __shared__ int scan_lds[kWaves];
  __shared__ int my_seg, my_tile;
  __shared__ int odd_tile;  // 1 + the diagonal tile found to hold a value that is not finite

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
  lo = __builtin_amdgcn_readfirstlane(lo);
  const int len = __builtin_amdgcn_readfirstlane(hi) - lo;
  const int r0 = __builtin_amdgcn_readfirstlane(my_tile) * kRows;
  const int w0 = r0 + wave * 32;  // this wave's first query
  const int query = w0 + col;
  const bool real = seg >= 1 && seg <= a.batch;

  f32x16 acc[kBlocks];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[i][j] = 0.f;
  // the running maximum (of the scores before scaling) and sum
  float m = kNegInf, l = 0.f;

  if (real) {
    // a negative scale goes into the queries' signs, so that the largest
    // product is the largest score; and no scale is 0, which would make NaN
    // of a masked score (weights differ from those of 0 by 1e-30)
    const float scale2 = fmaxf(fabsf(a.scale) * kLog2e, 1e-37f);
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
    bf16x8 qf[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      u32x4 w = {0, 0, 0, 0};
      if (query < len)
        w = *reinterpret_cast<const u32x4*>(a.q + (long long)(lo + query) * a.q_token +
                                            head * a.q_head + s * 16 + half * 8);
      qf[s] = __builtin_bit_cast(bf16x8, w ^ flip);
    }
    const uint16_t* kp = a.k + (long long)lo * a.k_token + kvh * a.k_head;
    const uint16_t* vp = a.v + (long long)lo * a.v_token + kvh * a.v_head;
    const int keys = min(len, r0 + kRows);  // that any query of the workgroup sees

    // Staging: load i of a wave fills 64 chunks, rows of kChunks, in LDS
    // order; a lane fetches the chunk that belongs at its place.  Rows past
    // the last key are past the resource's end and read as zeros.
    const int row_in = tid / kChunks, chunk_in = tid % kChunks;
    constexpr int kRowsPerLoad = kThreads / kChunks;
    const uint32_t k_off = (uint32_t)(row_in * a.k_token * 2), v_off = (uint32_t)(row_in * a.v_token * 2);
    const uint32_t lds0 = lds_dma::lds_addr(lds) + wave * 1024;
    auto stage = [&](const uint16_t* p, long long stride, uint32_t off, bool value, int block) __attribute__((always_inline)) {
      const int left = min(keys - block * 32, 32);
      const i32x4 rs = lds_dma::rsrc(p + (long long)block * 32 * stride,
                                     left > 0 ? (uint32_t)((left - 1) * (uint32_t)stride + D) * 2 : 0u);
      const uint32_t at = lds0 + ((value ? 4 : 0) + (block & 3)) * kBlockBytes;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = row_in + i * kRowsPerLoad;
        const int c = chunk_in ^ (value ? v_key<D>(r) : k_key<D>(r));
        lds_dma::dma16(rs, at + i * (kThreads * 16),
                       r < left ? off + (uint32_t)(i * kRowsPerLoad) * (uint32_t)stride * 2 + (c << 4)
                                : lds_dma::kSkip, 0);
      }
    };
    auto stage_k = [&](int block) __attribute__((always_inline)) { stage(kp, a.k_token, k_off, false, block); };
    auto stage_v = [&](int block) __attribute__((always_inline)) { stage(vp, a.v_token, v_off, true, block); };
    const int v_row = half * 4 + ((lane & 15) >> 2);

    // The steps of a block of 32 keys: its scores, the largest one, the
    // weights, their product with the values.  `block` (a constant) counts the
    // four blocks of the two tiles in LDS.
    float mx;
    auto scores = [&](auto block, f32x16& s) __attribute__((always_inline)) {
      const uint8_t* ks = lds + block * kBlockBytes;
#pragma unroll
      for (int j = 0; j < 16; ++j) s[j] = 0.f;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const bf16x8 kf = *reinterpret_cast<const bf16x8*>(
            ks + col * kRowBytes + (((2 * k + half) ^ k_key<D>(col)) << 4));
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[k], s, 0, 0, 0);
      }
    };
    // keys after the query, in the block that starts with the wave's first one
    auto hide = [&](f32x16& s) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if ((j & 3) + 8 * (j >> 2) + 4 * half > col) s[j] = kNegInf;
    };
    auto largest = [&](const f32x16& s) __attribute__((always_inline)) {
      float x = s[0];
#pragma unroll
      for (int j = 1; j < 16; ++j) x = fmaxf(x, s[j]);
      return half_max(x);
    };
    // The subtrahend follows the maximum only when that would let a weight
    // pass 2^kSlack: the outputs are then scaled down, which late blocks
    // almost never need.  A query's result depends on its own scores only.
    auto follow = [&]() __attribute__((always_inline)) {
      const bool grown = (mx - m) * scale2 > kSlack;
      if (__any(grown)) {
        const float alpha = grown ? __builtin_amdgcn_exp2f((m - mx) * scale2) : 1.f;
        m = grown ? mx : m;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) acc[i] *= alpha;
      }
    };
    auto weights = [&](const f32x16& s, bf16x8 (&pf)[2]) __attribute__((always_inline)) {
      const float ms = m == kNegInf ? 0.f : m * scale2;
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = __builtin_amdgcn_exp2f(fmaf(s[k * 8 + j], scale2, -ms));
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          sum0 += p[j];
          sum1 += p[j + 1];
        }
        pf[k] = __builtin_bit_cast(bf16x8, (u32x4){pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]),
                                                   pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7])});
      }
      l += sum0 + sum1;
    };
    auto add_values = [&](auto block, const bf16x8 (&pf)[2]) __attribute__((always_inline)) {
      const uint8_t* vs = lds + (4 + block) * kBlockBytes;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          u32x2 x[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = k * 16 + e * 8 + v_row;
            const int c = i * 4 + ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
            x[e] = lds_read_tr(vs + r * kRowBytes + ((c ^ v_key<D>(r)) << 4) + (lane & 1) * 8);
          }
          const bf16x8 vf = __builtin_bit_cast(bf16x8, (u32x4){x[0][0], x[0][1], x[1][0], x[1][1]});
          acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[k], acc[i], 0, 0, 0);
        }
    };
    auto add_odd = [&](int k0) __attribute__((always_inline)) {
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
    };

    // Takes the scores of a block through softmax and values while it computes
    // those of the next one: matrix and vector work of one wave that do not
    // wait for each other.
    auto step = [&](auto block, f32x16& s, f32x16& next) __attribute__((always_inline)) {
      follow();
      bf16x8 pf[2];
      scores(std::integral_constant<int, (block + 1) % 4>{}, next);
      weights(s, pf);
      add_values(block, pf);
      mx = largest(next);
    };
    // Landed after this: V of blocks u and u + 1, K of u + 1 and u + 2; every
    // wave is done with the blocks before those, whose places the next ones
    // take.
    auto turn = [&](int u) __attribute__((always_inline)) {
      lds_dma::wait_vmem<0>();
      lds_dma::lds_barrier();
      stage_v(u + 2);
      stage_v(u + 3);
      stage_k(u + 3);
      stage_k(u + 4);
    };
    constexpr std::integral_constant<int, 0> kB0;
    constexpr std::integral_constant<int, 1> kB1;
    constexpr std::integral_constant<int, 2> kB2;
    constexpr std::integral_constant<int, 3> kB3;
    f32x16 s0, s1;
    stage_k(0);
    stage_v(0);
    stage_v(1);
    stage_k(1);
    stage_k(2);
    lds_dma::wait_vmem<4 * kLoads>();
    lds_dma::lds_barrier();
    scores(kB0, s0);
    mx = largest(s0);
    // the blocks that all queries of the workgroup see whole
    const int whole = r0 / 32;
    for (int u = 0; u < whole; u += 4) {
      turn(u);
      step(kB0, s0, s1);
      step(kB1, s1, s0);
      turn(u + 2);
      step(kB2, s0, s1);
      step(kB3, s1, s0);
    }
    // the diagonal: a wave sees as many of its blocks as waves come before
    // it, and a part of one more
    auto diagonal = [&](auto block, f32x16& s, f32x16& next) __attribute__((always_inline)) {
      if (block < wave) {
        step(block, s, next);
      } else if (block == wave) {
        hide(s);
        mx = largest(s);
        follow();
        bf16x8 pf[2];
        weights(s, pf);
        add_values(block, pf);
      }
    };
    auto diagonal_tile = [&](auto block, auto block1) __attribute__((always_inline)) {
      turn(whole + block);
      uint8_t* vs = lds + (4 + block) * kBlockBytes;
      bool odd = false;
#pragma unroll
      for (int i = 0; i < 2 * kLoads; ++i)
        odd |= any_odd(*reinterpret_cast<const u32x4*>(vs + (i * kThreads + tid) * 16));
      if (odd) odd_tile = block + 1;
      lds_dma::lds_barrier();
      odd = odd_tile == block + 1;
      if (odd) {
        for (int x = tid; x < kKeys * D; x += kThreads) {
          uint16_t* w = reinterpret_cast<uint16_t*>(vs) + x;
          if ((*w & 0x7F80u) == 0x7F80u) *w = 0;
        }
        lds_dma::lds_barrier();
      }
      diagonal(block, s0, s1);
      diagonal(block1, s1, s0);
      if (odd && query < len) add_odd(r0 + block * 32);
    };
    diagonal_tile(kB0, kB1);
    if (keys > r0 + kKeys) diagonal_tile(kB2, kB3);
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
