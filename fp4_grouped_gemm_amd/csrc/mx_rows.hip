// MXFP4 products of few rows (decode): C = A B^T for the rows of each expert,
// or silu(A Bg^T) * (A Bu^T) for the gated ones, BF16 or MXFP4 out.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 with E2M1 operands takes MXFP4 as it is:
// lane (r, q) = (l % 16, l / 16) holds 32 codes of row r, block q of four, and
// that block's E8M0 code, so a block's scale rides in the lane that holds the
// block and FP32 sums come out without a separate dequantisation.
//
// A workgroup takes the columns of one expert, 16 or 32, and its eight waves
// take groups of 512 K in turn; the rows of an expert, found in scans of
// m_indices, run 16 or 32 at a time.  The weights are read once for these
// rows, straight into registers: 64 contiguous bytes of each of 16 rows a
// load.  The waves' partial sums meet in LDS and are added in the waves'
// order, so results do not depend on timing.
#include "mx.h"

#include <climits>

namespace fgg {
namespace mx_rows_detail {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kScan = 1024;  // m_indices entries compacted per scan

// Four blocks' scale codes at any multiple of 4 bytes.
typedef int i32x4a4 __attribute__((ext_vector_type(4), aligned(4)));

// One group of 512 K (four K = 128 products) of N fragments of 16 rows.
template <int N>
struct Group {
  i32x4 v[N][4];
  i32x4 s[N];
};

// Blocks of K = 128 past `have` load the last one there is again (and are not
// multiplied): nothing past a row's end is read.
template <int N, bool STREAM>
__device__ __forceinline__ void load(Group<N>& g, const uint8_t* const (&v)[N],
                                     const uint8_t* const (&s)[N], int ss, int have, int q) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const i32x4* p = reinterpret_cast<const i32x4*>(v[n] + (size_t)ss * 256 + min(j, have - 1) * 64 + q * 16);
      g.v[n][j] = STREAM ? __builtin_nontemporal_load(p) : *p;
    }
    const uint8_t* p = s[n] + (size_t)ss * 16;
    if (have == 4) {
      g.s[n] = *reinterpret_cast<const i32x4a4*>(p);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) g.s[n][j] = *reinterpret_cast<const int*>(p + 4 * min(j, have - 1));
    }
  }
}

template <int RB, int CB>
__device__ __forceinline__ void multiply(const Group<RB>& a, const Group<CB>& b, int have, int q,
                                         f32x4 (&acc)[RB][CB]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j < have) {
#pragma unroll
      for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int c = 0; c < CB; ++c) {
          const i32x4 x = b.v[c][j], y = a.v[r][j];
          acc[r][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              (i32x8){x[0], x[1], x[2], x[3], 0, 0, 0, 0}, (i32x8){y[0], y[1], y[2], y[3], 0, 0, 0, 0},
              acc[r][c], 4, 4, 0, (int)((uint32_t)b.s[c][j] >> (8 * q)), 0,
              (int)((uint32_t)a.s[r][j] >> (8 * q)));
        }
    }
  }
}

// Column of a workgroup's 16 CB that row r of its B fragment c holds.  With
// two fragments a lane's sums are then 8 consecutive columns: lane (r, q) holds
// row r of C at columns 4 q + t of each fragment, t < 4.
template <int CB>
__device__ __forceinline__ int column(int c, int r) {
  return CB == 1 ? r : 8 * (r >> 2) + 4 * c + (r & 3);
}

template <int RB, int CB, bool GATED>
__device__ __forceinline__ void chunk(const MxGemmArgs& a, const uint8_t* const (&bv)[CB * (GATED ? 2 : 1)],
                                      const uint8_t* const (&bs)[CB * (GATED ? 2 : 1)], const int* rows, int base,
                                      int c0, int count, int n0, float* red) {
  constexpr int F = CB * (GATED ? 2 : 1);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const size_t Kp = (size_t)a.K / 2, Ks = (size_t)a.K / 32;
  const auto row = [&](int i) { return rows ? rows[i] : base + i; };
  const uint8_t *av[RB], *as[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const size_t m = (size_t)row(min(c0 + 16 * i + r, count - 1));  // (past the last: not stored)
    av[i] = a.A + m * Kp;
    as[i] = a.a_scale + m * Ks;
  }
  f32x4 acc[RB][F];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int c = 0; c < F; ++c) acc[i][c] = (f32x4){0.f, 0.f, 0.f, 0.f};
  const int steps = a.K / 128, groups = (steps + 3) / 4;
  for (int ss = wave; ss < groups; ss += kWaves) {
    const int have = min(4, steps - 4 * ss);
    Group<F> gb;
    Group<RB> ga;
    load<F, true>(gb, bv, bs, ss, have, q);
    load<RB, false>(ga, av, as, ss, have, q);
    multiply<RB, F>(ga, gb, have, q, acc);
  }
  f32x4* mine = reinterpret_cast<f32x4*>(red) + wave * RB * F * 64 + lane;
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int c = 0; c < F; ++c) mine[(i * F + c) * 64] = acc[i][c];
  __syncthreads();
  if (wave < RB) {
    const f32x4* from = reinterpret_cast<const f32x4*>(red) + wave * F * 64 + lane;
    f32x4 sum[F];
#pragma unroll
    for (int c = 0; c < F; ++c) {
      sum[c] = from[c * 64];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) sum[c] += from[(w * RB * F + c) * 64];
    }
    float v[4 * CB];
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
      for (int t = 0; t < 4; ++t) v[4 * c + t] = GATED ? mx::gated(sum[c][t], sum[CB + c][t]) : sum[c][t];
    const int i = c0 + 16 * wave + r, n = n0 + 4 * CB * q;
    const bool store = i < count && n < a.N;
    const size_t m = (size_t)row(min(i, count - 1));
    if constexpr (CB == 2) {
      if (a.c_scale) {
        uint32_t top = mx::top8(v);
        top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
        const uint32_t code = mx::scale_code(top);
        const uint32_t word = code == 255u ? 0u : mx::codes8(v, mx::inverse(code));
        if (store) {
          *reinterpret_cast<uint32_t*>(a.C + m * (a.N / 2) + n / 2) = word;
          if (q == 0) a.c_scale[m * (a.N / 32) + n / 32] = (uint8_t)code;
        }
      } else if (store) {
        const uint2 lo = pack_bf16x4(v[0], v[1], v[2], v[3]), hi = pack_bf16x4(v[4], v[5], v[6], v[7]);
        *reinterpret_cast<uint4*>(a.C + (m * a.N + n) * 2) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    } else if (store) {
      *reinterpret_cast<uint2*>(a.C + (m * a.N + n) * 2) = pack_bf16x4(v[0], v[1], v[2], v[3]);
    }
  }
  __syncthreads();  // the sums are read before the next chunk's are written
}

template <int CB, bool GATED>
__global__ __launch_bounds__(kThreads) void mx_rows_kernel(const MxGemmArgs a, int nblk) {
  constexpr int F = CB * (GATED ? 2 : 1), kCols = 16 * CB;
  __shared__ __attribute__((aligned(16))) float red[kWaves * 2 * F * 256];
  __shared__ int rows[kScan];
  __shared__ int nrows;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = (blockIdx.x % nblk) * kCols, g = blockIdx.x / nblk;
  const size_t Kp = (size_t)a.K / 2, Ks = (size_t)a.K / 32;
  // this lane's row of each B fragment (columns past N: the last one, not stored)
  const uint8_t *bv[F], *bs[F];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const int n = min(n0 + column<CB>(f % CB, lane & 15), a.N - 1) + (f >= CB ? a.N : 0);
    const size_t b = (size_t)g * (GATED ? 2 : 1) * a.N + n;
    bv[f] = a.B + b * Kp;
    bs[f] = a.b_scale + b * Ks;
  }
  for (int scan0 = 0; scan0 < a.M; scan0 += kScan) {
    const int end = min(a.M, scan0 + kScan);
    int count = end - scan0;
    if (a.m_indices) {
      __syncthreads();  // the previous scan's rows are done with
      if (wave == 0) {
        count = 0;
        for (int i0 = scan0; i0 < end; i0 += 64) {
          const int i = i0 + lane;
          const int e = i < end ? a.m_indices[i] : g;
          const bool hit = i < end && e == g;
          const uint64_t mask = __ballot(hit);
          if (hit) rows[count + __popcll(mask & ((1ull << lane) - 1ull))] = i;
          count += __popcll(mask);
          // rows of no expert: zeros, written by expert 0's workgroups
          uint64_t bad = __ballot(g == 0 && (e < 0 || e >= a.G));
          while (bad) {
            const size_t m = (size_t)(i0 + __builtin_ctzll(bad));
            bad &= bad - 1;
            if (a.c_scale) {
              if (lane < kCols / 2 && n0 + 2 * lane < a.N) a.C[m * (a.N / 2) + n0 / 2 + lane] = 0;
              if (lane == 0) a.c_scale[m * (a.N / 32) + n0 / 32] = 0;
            } else if (lane < kCols && n0 + lane < a.N) {
              reinterpret_cast<uint16_t*>(a.C)[m * a.N + n0 + lane] = 0;
            }
          }
        }
        if (lane == 0) nrows = count;
      }
      __syncthreads();
      count = nrows;
    }
    const int* list = a.m_indices ? rows : nullptr;
    for (int c0 = 0; c0 < count; c0 += 32) {
      if (count - c0 > 16)
        chunk<2, CB, GATED>(a, bv, bs, list, scan0, c0, count, n0, red);
      else
        chunk<1, CB, GATED>(a, bv, bs, list, scan0, c0, count, n0, red);
    }
  }
}

template <int CB, bool GATED>
hipError_t launch(const MxGemmArgs& a, hipStream_t s) {
  const int nblk = (a.N + 16 * CB - 1) / (16 * CB);
  const long long grid = (long long)nblk * a.G;
  if (grid * kThreads > 0xFFFFFFFFLL) return hipErrorInvalidValue;
  hipLaunchKernelGGL((mx_rows_kernel<CB, GATED>), dim3((unsigned)grid), dim3(kThreads), 0, s, a, nblk);
  return hipGetLastError();
}

}  // namespace mx_rows_detail

hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t s) {
  using namespace mx_rows_detail;
  // 32 columns a workgroup, 16 where those would leave compute units idle
  const bool narrow = !a.c_scale && (long long)((a.N + 31) / 32) * a.G < a.num_cus;
  if (a.gated) return narrow ? launch<1, true>(a, s) : launch<2, true>(a, s);
  return narrow ? launch<1, false>(a, s) : launch<2, false>(a, s);
}

}  // namespace fgg
