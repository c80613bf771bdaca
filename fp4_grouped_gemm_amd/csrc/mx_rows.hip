// MXFP4 products of few rows (decode): C = A B^T for the rows of each expert,
// or silu(A Bg^T) * (A Bu^T) for the gated ones, BF16 or MXFP4 out.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 with E2M1 operands takes MXFP4 as it is:
// lane (r, q) = (l % 16, l / 16) holds 32 codes of row r and that block's E8M0
// code, so a block's scale rides in the lane that holds the block and FP32 sums
// come out without a separate dequantisation.
//
// With few rows the weights are the traffic, each byte used once, so the kernel
// is a stream of them: a wave owns 32 rows of B (of gated products 16 gate rows
// and the 16 up rows that go with them) over all of K, or a part of K where there
// are too few columns for all waves; and a ring of two or three steps of 256 K in
// LDS of its own, which it fills by direct loads of whole lines (these stream
// faster than loads into registers: 128 rows over 8 experts of 8192 columns and
// K 55 us against 95) and reads without waiting for any other wave.  The rows of
// A that go with an expert are found in scans of m_indices by each wave for
// itself and come through the same ring, 16 or 32 at a time.  The waves' sums meet
// in LDS at the end and are added in the waves' order, so results do not depend
// on timing.
//
// Measured: 8 experts of 8192 x 8192 (285 MB with scale codes), 8 rows 45 us (6.3
// TB/s), 128 rows 55 us (5.2 TB/s; a copy on this card reaches 4.6): memory bounds
// it, and the rows of A that each wave reads for itself.  64 rows of B a wave, with
// half of that traffic, gained nothing (57 us against 57 at the time) and slowed
// smaller products; 16 rows nothing for one token (5.9 us against 5.8 at 4096 x
// 4096, where calls of the smallest products follow each other every 4 us).
#include "mx.h"
#include "mx_rule.h"
#include "offsets.h"

#include <climits>

namespace fgg {
namespace mx_rows_detail {

using namespace lds_dma;

constexpr int kScan = 1024;       // m_indices entries compacted per scan
constexpr int kNoStep = 1 << 24;  // of 256 K: past the end of every operand's

constexpr int F = 2;  // fragments of 16 rows of B a wave: 32 columns, or 16 gate and 16 up rows

template <bool GATED_>
struct Cfg {
  static constexpr int W = 4;  // waves a workgroup; two workgroups a CU
  static constexpr bool GATED = GATED_;
  static constexpr int THREADS = 64 * W;
  static constexpr int COLS = GATED ? 16 : 16 * F;  // columns of C a wave's rows of B make
};

template <class V>
__device__ __forceinline__ V lds_read(uint32_t at) {
  return *reinterpret_cast<__attribute__((address_space(3))) const V*>(at);
}

// dma16 of bytes that are not read again: they leave the caches to what is (A
// and the lines that hold scale codes, 16 bytes a row at a time).
__device__ __forceinline__ void dma16_once(i32x4 rs, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds" ::"s"(lds), "v"(voff), "s"(rs), "s"(soff)
               : "memory", "m0");
}

// A wave's ring with 16 RB rows of A: three steps of 16 rows, or two of 32, and
// the scale codes (16 bytes a row) of twice two steps.
template <class T, int RB>
struct Ring {
  static constexpr int N = RB == 1 ? 3 : 2, SLOT = F * 2048 + RB * 2048;
  static constexpr int CODES = N * SLOT, SCALES = F * 256 + RB * 256;
  static constexpr int BYTES = CODES + 2 * SCALES;
  static constexpr int LOADS = 2 * F + 2 * RB, SCALE_LOADS = (T::GATED ? 2 : 1) + 1;
};
template <class T>
constexpr int ring_bytes() {
  return Ring<T, 1>::BYTES > Ring<T, 2>::BYTES ? Ring<T, 1>::BYTES : Ring<T, 2>::BYTES;
}

// A wave's operands: B's rows (of gated products gate and up), and A.
struct Stream {
  i32x4 rb[2], rsb[2], ra, rsa;
  uint32_t a_off[4];      // of the four loads of A's 32 rows (kSkip: no such row)
  uint32_t as_off;        // scale codes of A's row `lane`
  uint32_t Kp, Ks;
  int K128;
};

// Step k into its slot: every step issues the same loads, those past the
// last step of nothing (zeros, no memory is read), as the second half of an odd
// multiple of 128 is.
template <class T, int RB, bool ONCE>
__device__ __forceinline__ void load_step(const Stream& s, uint32_t slot, int k, int lane) {
  const uint32_t at = (uint32_t)k * 128u;
  const bool there = 2 * k < s.K128;
#pragma unroll
  for (int i = 0; i < 2 * F; ++i) {
    // (the rows' swizzle depends on which half of 16 rows they are)
    const int chunk = (lane & 7) ^ off::fp8_swz_key(((i & 1) << 3) + (lane >> 3));
    i32x4 r = s.rb[T::GATED ? i >> 1 : 0];
    r[2] = there ? r[2] : 0;
    const uint32_t row = (uint32_t)((T::GATED ? (i & 1) * 8 : i * 8) + (lane >> 3));
    const uint32_t none = 2 * k + 1 == s.K128 && chunk >= 4 ? kSkip : 0u;
    const uint32_t from = (row * s.Kp + (uint32_t)chunk * 16u) | none;
    if constexpr (ONCE)
      dma16_once(r, slot + i * 1024, from, at);
    else
      dma16(r, slot + i * 1024, from, at);
  }
  i32x4 r = s.ra;
  r[2] = there ? r[2] : 0;
#pragma unroll
  for (int i = 0; i < 2 * RB; ++i) {
    const int chunk = (lane & 7) ^ off::fp8_swz_key(((i & 1) << 3) + (lane >> 3));
    const uint32_t none = 2 * k + 1 == s.K128 && chunk >= 4 ? kSkip : 0u;
    dma16(r, slot + F * 2048 + i * 1024, (s.a_off[i] + (uint32_t)chunk * 16u) | none, at);
  }
}
// The scale codes of steps k and k + 1, k even, into buffer b % 2, a lane a row.  A
// row whose end lies among them reads on into the next row: the reads below
// leave those codes out.
template <class T, int RB>
__device__ __forceinline__ void load_scales(const Stream& s, uint32_t ring, int b, int k, int lane) {
  const uint32_t to = ring + Ring<T, RB>::CODES + (b & 1) * Ring<T, RB>::SCALES;
  const uint32_t at = (uint32_t)k * 8u;
  const bool there = 2 * k < s.K128;
  if (lane < (T::GATED ? 16 : 16 * F)) {
#pragma unroll
    for (int g = 0; g < (T::GATED ? 2 : 1); ++g) {
      i32x4 r = s.rsb[g];
      r[2] = there ? r[2] : 0;
      dma16(r, to + g * 256, (uint32_t)lane * s.Ks + at, 0);
    }
  }
  if (lane < 16 * RB) {
    i32x4 r = s.rsa;
    r[2] = there ? r[2] : 0;
    dma16(r, to + F * 256, s.as_off == kSkip ? kSkip : s.as_off + at, 0);
  }
}
// Lane (r, q)'s codes of blocks 2 q and 2 q + 1 of the i-th step, k, and their
// scale codes in bytes 0 and 1.
template <int RB>
struct Frags {
  i32x4 b[F][2], a[RB][2];
  int sb[F], sa[RB];
};
template <class T, int RB>
__device__ __forceinline__ void read(Frags<RB>& f, const Stream& s, uint32_t ring, uint32_t slot, int i, int k, int lane) {
  const int r = lane & 15, q = lane >> 4;
  const uint32_t sc = ring + Ring<T, RB>::CODES + ((i >> 1) & 1) * Ring<T, RB>::SCALES + (i & 1) * 8 + 2 * q;
  // (past the end of K: codes of zero, so that no NaN meets the zeros there)
  const int mask = 2 * k + (q >> 1) < s.K128 ? 0xFFFF : 0;
#pragma unroll
  for (int j = 0; j < F; ++j) {
#pragma unroll
    for (int h = 0; h < 2; ++h) f.b[j][h] = lds_read<i32x4>(slot + j * 2048 + off::fp8_lds_off(r, 2 * q + h));
    f.sb[j] = lds_read<uint16_t>(sc + (j * 16 + r) * 16) & mask;
  }
#pragma unroll
  for (int m = 0; m < RB; ++m) {
#pragma unroll
    for (int h = 0; h < 2; ++h) f.a[m][h] = lds_read<i32x4>(slot + (F + m) * 2048 + off::fp8_lds_off(r, 2 * q + h));
    f.sa[m] = lds_read<uint16_t>(sc + ((F + m) * 16 + r) * 16) & mask;
  }
}

template <int H>
__device__ __forceinline__ f32x4 multiply(i32x4 b, int sb, i32x4 a, int sa, f32x4 acc) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4((i32x8){b[0], b[1], b[2], b[3], 0, 0, 0, 0},
                                                          (i32x8){a[0], a[1], a[2], a[3], 0, 0, 0, 0}, acc, 4, 4, H, sb,
                                                          H, sa);
}

// Steps [k0, k0 + n) of 16 RB rows of A, k0 and n even, from the first + turn
// on and round.  Waves that begin at different places of K do not all ask the
// same memory channels at once where the rows' length is a power of two (8192
// columns of 8192 K of each of eight experts: 55 us against 59, and 57 against
// 66 where one wave takes all of K).
template <class T, int RB, bool ONCE>
__device__ __forceinline__ void stream(const Stream& s, uint32_t ring, int k0, int n, int turn, int lane,
                                       f32x4 (&acc)[2][F]) {
  using R = Ring<T, RB>;
  // The i-th step (past the last one, one past the end of K).
  const auto step = [&](int i) {
    return __builtin_amdgcn_readfirstlane(i >= n ? kNoStep : k0 + (i + turn >= n ? i + turn - n : i + turn));
  };
  load_scales<T, RB>(s, ring, 0, step(0), lane);
#pragma unroll
  for (int i = 0; i < R::N; ++i) {
    // (second of the scale codes' loads before the last step's, as below)
    if (i == R::N - 1) load_scales<T, RB>(s, ring, 1, step(2), lane);
    load_step<T, RB, ONCE>(s, ring + i * R::SLOT, step(i), lane);
  }
  uint32_t slot = ring;
  for (int i = 0; i < n; ++i) {
    // What may be on its way: the steps after this one; and scale codes, which
    // are asked for after a step is read that is the second of two, before the
    // step that takes its slot.
    if (R::N == 3 || i % 2 == 0)
      wait_vmem<(R::N - 1) * R::LOADS + R::SCALE_LOADS>();
    else
      wait_vmem<(R::N - 1) * R::LOADS>();
    Frags<RB> f;
    read<T, RB>(f, s, ring, slot, i, step(i), lane);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read, before the slot is filled again
    if (i % 2) load_scales<T, RB>(s, ring, i / 2, step(i + 3), lane);
    load_step<T, RB, ONCE>(s, slot, step(i + R::N), lane);
    slot = slot + R::SLOT == ring + R::N * R::SLOT ? ring : slot + R::SLOT;
#pragma unroll
    for (int m = 0; m < RB; ++m)
#pragma unroll
      for (int j = 0; j < F; ++j) acc[m][j] = multiply<0>(f.b[j][0], f.sb[j], f.a[m][0], f.sa[m], acc[m][j]);
#pragma unroll
    for (int m = 0; m < RB; ++m)
#pragma unroll
      for (int j = 0; j < F; ++j) acc[m][j] = multiply<1>(f.b[j][1], f.sb[j], f.a[m][1], f.sa[m], acc[m][j]);
  }
  wait_vmem<0>();  // (loads of nothing, which write zeros to the ring)
}

// Rows c0 .. c0 + 16 RB of the expert's (numbered from `base`): the waves' sums,
// and from them C.
template <class T, int RB, bool ONCE>
__device__ __forceinline__ void chunk(const MxGemmArgs& a, Stream& s, uint8_t* lds, const uint16_t* rows, int base, int c0, int count,
                                      int n0, int ksplit, int wave, int lane) {
  const uint32_t ring = lds_addr(lds) + wave * ring_bytes<T>();
  const auto row = [&](int i) { return rows ? (int)rows[i] : i; };
#pragma unroll
  for (int i = 0; i < 2 * RB; ++i) {
    const int c = c0 + i * 8 + (lane >> 3);
    s.a_off[i] = c < count ? (uint32_t)row(c) * s.Kp : kSkip;
  }
  s.as_off = c0 + lane < count ? (uint32_t)row(c0 + lane) * s.Ks : kSkip;
  f32x4 acc[2][F];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
  // this wave's part of K: an even number of steps
  const int pairs = (s.K128 + 3) / 4, per = (pairs + ksplit - 1) / ksplit;
  const int p0 = (wave % ksplit) * per, np = __builtin_amdgcn_readfirstlane(min(per, pairs - p0));
  if (np > 0) stream<T, RB, ONCE>(s, ring, 2 * p0, 2 * np, 2 * ((int)((blockIdx.x * 5 + wave) & 0xFFFF) % np), lane, acc);
  f32x4* mine = reinterpret_cast<f32x4*>(lds + wave * ring_bytes<T>()) + lane;
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) mine[(i * F + j) * 64] = acc[i][j];
  __syncthreads();
  // a thread takes eight columns of a row: four lanes an MXFP4 block
  const int groups = T::W / ksplit * T::COLS / 8;
  for (int t = wave * 64 + lane; t < 16 * RB * groups; t += T::THREADS) {
    const int m = t / groups, c = t % groups * 8;
    const int w = c / T::COLS * ksplit, f = T::GATED ? 0 : c % T::COLS / 16, q = c % 16 / 4;
    const auto sum = [&](int frag, int quad) {
      f32x4 x = {0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < ksplit; ++k)
        x += reinterpret_cast<const f32x4*>(lds + (w + k) * ring_bytes<T>())[((m >> 4) * F + frag) * 64 + quad * 16 + (m & 15)];
      return x;
    };
    float v[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 x = sum(f, q + h);
      if constexpr (T::GATED) {
        const f32x4 up = sum(1, q + h);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * h + i] = mx::gated(x[i], up[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * h + i] = x[i];
      }
    }
    const int n = n0 + c;
    const bool store = c0 + m < count && n < a.N;
    const size_t to = store ? (size_t)(base + row(c0 + m)) * a.N + n : 0;
    if (T::GATED && a.c_scale) {
      uint32_t top = mx::top8(v);
      top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
      top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
      const uint32_t code = mx::scale_code(top);
      const uint32_t word = code == 255u ? 0u : mx::codes8(v, mx::inverse(code));
      if (store) {
        *reinterpret_cast<uint32_t*>(a.C + to / 2) = word;
        if (c % 32 == 0) a.c_scale[to / 32] = (uint8_t)code;
      }
    } else if (store) {
      const uint2 lo = pack_bf16x4(v[0], v[1], v[2], v[3]), hi = pack_bf16x4(v[4], v[5], v[6], v[7]);
      *reinterpret_cast<uint4*>(a.C + to * 2) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
  __syncthreads();  // the sums and the rows are done with
}

template <class T>
__global__ __launch_bounds__(T::THREADS, 2) void mx_rows_kernel(const MxGemmArgs a, int nblk, int ksplit, bool by_row) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::W * ring_bytes<T>()];
  __shared__ uint16_t rows[kScan];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int cols = T::W / ksplit * T::COLS;  // of the workgroup
  const int n0 = (int)(blockIdx.x % nblk) * cols;
  int g = (int)(blockIdx.x / nblk);
  const auto clear = [&](int m) {  // a row of no expert: zeros
    for (int c = 8 * lane; c < cols && n0 + c < a.N; c += 512) {
      const size_t to = (size_t)m * a.N + n0 + c;
      if (T::GATED && a.c_scale) {
        *reinterpret_cast<uint32_t*>(a.C + to / 2) = 0u;
        if (c % 32 == 0) a.c_scale[to / 32] = 0;
      } else {
        *reinterpret_cast<uint4*>(a.C + to * 2) = make_uint4(0, 0, 0, 0);
      }
    }
  };
  int found = 0;
  if (by_row) {
    // The g-th of the experts that have rows (none, -1, among them).
    const int e = lane < a.M ? a.m_indices[lane] : -1, key = e >= 0 && e < a.G ? e : -1;
    bool first = lane < a.M;
    for (int j = 0; j < a.M; ++j) first &= j >= lane || __builtin_amdgcn_readlane(key, j) != key;
    uint64_t mask = __ballot(first);
    if (g >= __popcll(mask)) return;
    for (int j = 0; j < g; ++j) mask &= mask - 1;
    g = __builtin_amdgcn_readlane(key, __builtin_ctzll(mask));
    if (g < 0) {
      for (uint64_t none = __ballot(lane < a.M && key < 0); none && wave == 0; none &= none - 1) clear(__builtin_ctzll(none));
      return;
    }
    const uint64_t mine = __ballot(lane < a.M && key == g);
    if (lane < a.M && key == g) rows[__popcll(mine & ((1ull << lane) - 1ull))] = (uint16_t)lane;
    found = __popcll(mine);
  }
  Stream s;
  s.Kp = (uint32_t)a.K / 2;
  s.Ks = (uint32_t)a.K / 32;
  s.K128 = a.K / 128;
  // this wave's rows of B, those past the last column of nothing
  const int n = n0 + wave / ksplit * T::COLS, left = min(T::COLS, a.N - n);
  const uint32_t there = left > 0 ? (uint32_t)left : 0u;
#pragma unroll
  for (int h = 0; h < (T::GATED ? 2 : 1); ++h) {
    const size_t b = ((size_t)g * (T::GATED ? 2 : 1) + h) * a.N + n;
    s.rb[h] = rsrc(a.B + b * s.Kp, there * s.Kp);
    s.rsb[h] = rsrc(a.b_scale + b * s.Ks, there * s.Ks);
  }
  for (int scan0 = 0; scan0 < a.M; scan0 += kScan) {
    const int end = min(a.M, scan0 + kScan);
    int count = end - scan0;
    s.ra = rsrc(a.A + (size_t)scan0 * s.Kp, (uint32_t)count * s.Kp);
    s.rsa = rsrc(a.a_scale + (size_t)scan0 * s.Ks, (uint32_t)count * s.Ks);
    if (by_row) {
      count = found;
    } else if (a.m_indices) {
      // Every wave makes the whole list (the same values in the same places),
      // from loads that are all on their way together.
      int e[kScan / 64];
#pragma unroll
      for (int i = 0; i < kScan / 64; ++i) {
        const int m = scan0 + i * 64 + lane;
        e[i] = m < end ? a.m_indices[m] : INT_MAX;
      }
      count = 0;
#pragma unroll
      for (int i = 0; i < kScan / 64; ++i) {
        if (scan0 + i * 64 >= end) break;
        const int m = scan0 + i * 64 + lane;
        const bool hit = e[i] == g;
        const uint64_t mask = __ballot(hit);
        if (hit) rows[count + __popcll(mask & ((1ull << lane) - 1ull))] = (uint16_t)(m - scan0);
        count += __popcll(mask);
        // (rows of no expert are left to expert 0's workgroups)
        if (g == 0 && wave == 0)
          for (uint64_t none = __ballot(m < end && (e[i] < 0 || e[i] >= a.G)); none; none &= none - 1)
            clear(scan0 + i * 64 + __builtin_ctzll(none));
      }
    }
    const uint16_t* list = a.m_indices ? rows : nullptr;
    // Weights that are read once are asked for as such: 8 experts of 8192 columns
    // and K, 1 and 16 rows each, 45 and 55 us against 50 and 58; one row of 28672
    // columns, 4096 K, 13.8 against 14.5; but 64 rows each, two passes over the
    // weights, 66 against 57.  Where K is split over four waves the weights are few,
    // and may be in a cache from an earlier call: 4096 x 4096 5.9 against 5.6.
    const bool once = count <= 32 && a.M <= kScan && ksplit < 4;
    for (int c0 = 0; c0 < count; c0 += 32) {
      const bool two = count - c0 > 16;
      if (once && two)
        chunk<T, 2, true>(a, s, lds, list, scan0, c0, count, n0, ksplit, wave, lane);
      else if (once)
        chunk<T, 1, true>(a, s, lds, list, scan0, c0, count, n0, ksplit, wave, lane);
      else if (two)
        chunk<T, 2, false>(a, s, lds, list, scan0, c0, count, n0, ksplit, wave, lane);
      else
        chunk<T, 1, false>(a, s, lds, list, scan0, c0, count, n0, ksplit, wave, lane);
    }
  }
}

template <class T>
hipError_t launch(const MxGemmArgs& a, int ksplit, hipStream_t s) {
  const int cols = T::W / ksplit * T::COLS, nblk = (a.N + cols - 1) / cols;
  // No more experts have rows than there are rows (two rows of eight experts,
  // 2048 gated columns of 4096 K: 8.1 us against 10.5 with a workgroup for
  // every expert; where the workgroups fit the card at once it is the same).
  const bool by_row = a.m_indices && a.M <= 64 && a.M < a.G;
  const long long grid = (long long)nblk * (by_row ? a.M : a.G);
  if (grid * T::THREADS > 0xFFFFFFFFLL) return hipErrorInvalidValue;
  hipLaunchKernelGGL(mx_rows_kernel<T>, dim3((unsigned)grid), dim3(T::THREADS), 0, s, a, nblk, ksplit, by_row);
  return hipGetLastError();
}

}  // namespace mx_rows_detail

hipError_t launch_mx_rows(const MxGemmArgs& a, hipStream_t s) {
  using namespace mx_rows_detail;
  static_assert(Cfg<true>::COLS == mx::rows_columns(true) && Cfg<false>::COLS == mx::rows_columns(false), "the rule's columns");
  const int ksplit = mx::rows_ksplit(a.M, a.N, a.G, a.gated, a.c_scale != nullptr, a.num_cus);
  return a.gated ? launch<Cfg<true>>(a, ksplit, s) : launch<Cfg<false>>(a, ksplit, s);
}

}  // namespace fgg
