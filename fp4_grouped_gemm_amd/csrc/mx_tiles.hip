// MXFP4 products of many rows (prompts): C = A B^T for rows routed to experts,
// or silu(A Bg^T) * (A Bu^T) for the gated ones, BF16 or MXFP4 out.
//
// A work tile is a span of up to BM rows and BN rows of B (columns of C, or for
// gated products the gate and up rows of BN / 2 columns).  Where the rows come
// in runs of one expert, each workgroup finds the runs in m_indices and cuts
// each into spans of its own (rows of no expert are in none: the workgroups share
// out their zeros row by row; 8 experts of 4096 columns and K, 600 rows in 1024
// places each, 74 us against 100 with tiles of zeros); else the spans are windows
// of BM rows, which may hold rows of several experts, and the workgroup runs one
// pass of the K loop for each of them, storing that expert's rows.
//
// K steps of 256 values are 128 bytes a row, a whole cache line, staged in LDS
// by direct loads while the step before is multiplied; 16-byte chunks (32
// codes, a block) are XOR-swizzled by row so that reads of codes meet no bank
// conflict; the scale codes' reads, two bytes of each of 16 rows 16 bytes apart, meet
// two cycles of it each (which is all that is counted: 4.0 million for the 2.0
// million reads of the first case below, 4% of its time).  v_mfma_scale_f32_16x16x128_f8f6f4 takes a lane's 32
// codes and their scale code; which 32 of a step lane (r, q) = (l % 16, l / 16) takes is free as
// long as A and B agree: blocks 2 q and 2 q + 1, for the step's two products,
// so that a lane's codes and its two scale bytes are each contiguous.  Scale
// codes are staged for two steps at a time, 16 bytes a row.
//
// B's rows are dealt to the tile's LDS rows so that a lane's sums are eight
// consecutive columns of a row of C (16 bytes of BF16, or a quarter of an
// MXFP4 block), and so that gate and up of a column are in the same lane.
//
// Measured: 2048 rows, 36864 columns, 4608 K 191 us (3.6 PFLOP/s); 4096 rows,
// columns and K 43 us; 5554 rows of 8 experts, 2048 gated columns, 7168 K 127 us.
// The matrix instruction alone sustains 7.0 PFLOP/s with random operands (power:
// the clock falls from 2.4 to 2.0 GHz; its 32 x 32 x 64 form 6.3).  A step of 256 x
// 256 tiles takes 1.7 to 2.1 us, of which 1.1 are matrix instructions; without its
// loads 1.2.  Of 128 x 128 tiles, one workgroup a CU: 0.8 us, without what its loads
// bring 0.6, without the loads 0.43, 0.25 of that matrix instructions: reads and
// writes of LDS come next, then the latency of the loads.  Built and slower or no
// faster: 32 x 32 x 64 instructions, 128 x 128 products a wave (spills, with the sums
// in vector registers; in accumulation registers not tried), three
// stages of 128 x 256 (79 us against 87 for 55 rows of each of 8 experts, but 24
// against 19 for 512 rows of 4096 columns and K), steps asked for in L2 ahead.
#include "mx.h"
#include "mx_layout.h"
#include "mx_rule.h"
#include "offsets.h"

#include <algorithm>
#include <climits>

namespace fgg {
namespace mx_tiles_detail {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

using namespace lds_dma;

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, bool GATED_>
struct Cfg {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
  static constexpr bool GATED = GATED_;
  static constexpr int WAVES = WAVES_M * WAVES_N, THREADS = 64 * WAVES;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;  // rows of A and of B a wave multiplies
  static constexpr int TM = WM / 16, TN = WN / 16;
  static constexpr int COLS = GATED ? BN / 2 : BN;            // columns of C a tile holds
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;  // of a K step's tiles
  static constexpr int A_LOADS = BM / 8 / WAVES, B_LOADS = BN / 8 / WAVES;      // 8 rows a load
  static constexpr int SCALES = (BM + BN) * 16;               // bytes of two steps' scale codes
  static constexpr int WG_PER_CU = 160 * 1024 / (2 * (A_BYTES + B_BYTES + SCALES) + 4096);
  static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0, "load split");
  static_assert(BM + BN == 64 * WAVES && BM % 64 == 0 && COLS % 64 == 0, "a wave stages 64 rows' scale codes");
  static_assert(WAVES == 4 || WAVES == 8, "what of a load's place depends on its wave");
  static_assert(WM == 64 && BM <= 512 && WN % 64 == 0 && TM <= 2 * TN - 4, "tile shape");
};

// This lane's number, found anew: nothing that is computed from it can be kept
// in registers from one call to the next.
__device__ __forceinline__ int fresh_lane() {
  int l;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
  return l;
}

// Two steps of A's tile, then two of B's, then two chunks of scale codes (each
// of two steps, 16 bytes a row: the window's rows, then B's).  What a wave
// reads of either operand lies within the 64 KB that a read's constant offset
// spans, so one register holds the place of all its reads.
template <class T>
struct Lds {
  static constexpr int A = 0, B = 2 * T::A_BYTES, SC = B + 2 * T::B_BYTES, BYTES = SC + 2 * T::SCALES;
  static_assert(2 * T::A_BYTES <= 65536 && 2 * T::B_BYTES <= 65536, "a read's constant offset");
};

template <class V>
__device__ __forceinline__ V lds_read(uint32_t at) {
  return *reinterpret_cast<__attribute__((address_space(3))) const V*>(at);
}

template <class T>
struct Pass {
  i32x4 ra;  // A, the window's rows
  // B, the tile's rows of the expert.  Of gated products a load holds gate rows
  // or up rows, by its wave, or with four waves by its number.
  static constexpr int HALVES = T::GATED && T::WAVES == 4 ? 2 : 1;
  i32x4 rb[HALVES];
  i32x4 rs;               // a_scale or b_scale: the 64 rows whose scale codes this wave stages
  uint32_t lds;           // address of the stages
  uint32_t a_off, b_off;  // this lane's part of a load's offset
  uint32_t far;           // kSkip in lanes whose chunk is in a step's second half
  uint32_t a_at[2], b_at[2], sa_at, sb_at;  // where this lane reads codes (by half) and scale codes
  uint32_t sc_next;       // the scale codes' buffer that is filled, SCALES or 0
  uint32_t Kp, Ks;
  int K128;               // K / 128
  uint64_t a_groups;      // 8-row groups of the window with a row of this pass
  f32x4 acc[T::TM][T::TN];

  // Lane l of a load fills chunk l % 8 of its row l / 8 in LDS.
  __device__ __forceinline__ static int chunk_of(int lane, int wave) {
    return (lane & 7) ^ off::fp8_swz_key(((wave & 1) << 3) + (lane >> 3));
  }
  __device__ __forceinline__ void init(const MxGemmArgs& a, const void* stages, int lane, int wave, int wm, int wn) {
    Kp = (uint32_t)a.K / 2;
    Ks = (uint32_t)a.K / 32;
    K128 = a.K / 128;
    sc_next = 0;
    lds = lds_addr(stages);
    const uint32_t chunk = (uint32_t)chunk_of(lane, wave) * 16u;
    far = chunk >= 64u ? kSkip : 0u;
    a_off = (uint32_t)(wave * 8 + (lane >> 3)) * Kp + chunk;
    b_off = (uint32_t)mx::tile_column(wave, lane >> 3, T::GATED) * Kp + chunk;
    const int r = lane & 15, q = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      a_at[h] = lds + Lds<T>::A + wm * T::WM * 128 + off::fp8_lds_off(r, 2 * q + h);
      b_at[h] = lds + Lds<T>::B + wn * T::WN * 128 + off::fp8_lds_off(r, 2 * q + h);
    }
    sa_at = lds + Lds<T>::SC + (wm * T::WM + r) * 16 + 2 * q;
    sb_at = lds + Lds<T>::SC + (T::BM + wn * T::WN / (T::GATED ? 2 : 1) + r) * 16 + 2 * q;
    asm volatile("" : "+v"(a_off), "+v"(b_off), "+v"(far), "+v"(a_at[0]), "+v"(a_at[1]), "+v"(b_at[0]), "+v"(b_at[1]), "+v"(sa_at),
                 "+v"(sb_at));
  }

  // Load s of step k into the stage of parity P.  Every wave issues the same
  // number of loads at every step: those of row groups without a row of the
  // pass, and of steps past the last, go past the buffer's end (zeros, no
  // memory is read), and so does the second half of the last step of a K that
  // is an odd multiple of 128.  (The steps are opaque, so that their sums with
  // the offsets are not kept in registers over the K loop.)
  __device__ __forceinline__ i32x4 until_end(i32x4 r, int k) const {
    r[2] = 2 * k < K128 ? r[2] : 0;
    return r;
  }
  __device__ __forceinline__ uint32_t half_only(int k) const { return 2 * k + 1 == K128 ? far : 0u; }
  template <int P>
  __device__ __forceinline__ void load_a(int s, int k, int wave) const {
    const int b = s * T::WAVES + wave;
    uint32_t step = (a_groups >> b) & 1 ? (uint32_t)(s * T::WAVES * 8) * Kp : kSkip;
    asm volatile("" : "+s"(step));
    dma16(until_end(ra, k), lds + Lds<T>::A + P * T::A_BYTES + b * 1024, (a_off + step) | half_only(k), (uint32_t)k * 128u);
  }
  template <int P>
  __device__ __forceinline__ void load_b(int s, int k, int wave) const {
    uint32_t step = (uint32_t)mx::tile_step(s, T::WAVES, T::GATED) * Kp;
    asm volatile("" : "+s"(step));
    dma16(until_end(rb[HALVES > 1 ? mx::tile_half(s * T::WAVES, true) : 0], k),
          lds + Lds<T>::B + P * T::B_BYTES + (s * T::WAVES + wave) * 1024, (b_off + step) | half_only(k), (uint32_t)k * 128u);
  }
  // The scale codes of steps 2 c and 2 c + 1 into the buffer that the reads do
  // not go to, 16 bytes a row: a lane a row, or where the row ends among them
  // four lanes a row, zeros past its end.  Of B a wave's 64 rows lie as their
  // subtiles do (mx::tile_column), so that the 16 rows of one are read without
  // a bank conflict.
  __device__ __forceinline__ void load_scales(int c, int wave) const {
    const int lane = fresh_lane();
    const uint32_t to = lds + Lds<T>::SC + sc_next + wave * 1024;
    const auto row = [&](int p) {
      const int r = wave * 64 < T::BM ? p : mx::tile_column(p >> 3, p & 7, false);
      uint32_t at;  // (Ks in a scalar register: held in a vector one it would be spilled)
      asm("v_mul_u32_u24 %0, %1, %2" : "=v"(at) : "s"(Ks), "v"(r));
      return at;
    };
    if (4 * c + 4 <= K128) {
      dma16(rs, to, row(lane), (uint32_t)c * 16u);
    } else {
      const bool past = 4 * c + (lane & 3) >= K128;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        dma4(rs, to + s * 256, past ? kSkip : row(s * 16 + (lane >> 2)) + (uint32_t)(lane & 3) * 4u, (uint32_t)c * 16u);
    }
  }
  // The reads go on to the next two steps' scale codes.
  __device__ __forceinline__ void flip_scales() {
    const uint32_t by = sc_next ? (uint32_t)T::SCALES : 0u - (uint32_t)T::SCALES;
    sa_at += by;
    sb_at += by;
    sc_next = (uint32_t)T::SCALES - sc_next;
  }
  __device__ __forceinline__ void set_expert(const MxGemmArgs& a, int e, int row0, int col0, int wave) {
    const size_t row = (size_t)e * (T::GATED ? 2 : 1) * a.N + col0;
    const uint32_t rows = (uint32_t)min(T::COLS, a.N - col0);
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      const int half = HALVES > 1 ? h : mx::tile_half(wave, T::GATED);
      rb[h] = rsrc(a.B + (row + (size_t)half * a.N) * Kp, rows * Kp);
    }
    // scale rows in LDS: the window's, then the tile's columns (gate, then up)
    const int r = wave * 64, b = r - T::BM, half = b >= T::COLS ? 1 : 0, n = b - half * T::COLS;
    const uint8_t* from = r < T::BM ? a.a_scale + (size_t)(row0 + r) * Ks
                                    : a.b_scale + (row + (size_t)half * a.N + n) * Ks;
    const int left = r < T::BM ? a.M - row0 - r : (int)rows - n;
    rs = rsrc(from, left <= 0 ? 0u : left < 64 ? (uint32_t)left * Ks : 64u * Ks);
#pragma unroll
    for (int i = 0; i < 4; ++i) rs[i] = __builtin_amdgcn_readfirstlane(rs[i]);
  }

  // Fragments of half h of a step of parity P: lane (r, q) holds the 32 codes
  // of block 2 q + h of row r.  The scale codes of blocks 2 q and 2 q + 1 come
  // in bytes 0 and 1.
  template <int H, int P>
  __device__ __forceinline__ i32x4 a_codes(int i) const {
    return lds_read<i32x4>(a_at[H] + P * T::A_BYTES + i * 2048);
  }
  template <int H, int P>
  __device__ __forceinline__ i32x4 b_codes(int j) const {
    return lds_read<i32x4>(b_at[H] + P * T::B_BYTES + j * 2048);
  }
  template <int P>
  __device__ __forceinline__ int a_scales(int i) const {
    return lds_read<uint16_t>(sa_at + P * 8 + i * 256);
  }
  template <int P>
  __device__ __forceinline__ int b_scales(int j) const {
    // (gate columns' rows lie before up columns')
    const int row = T::GATED ? (j >> 2) * 32 + (j & 1) * 16 + ((j >> 1) & 1) * T::COLS : j * 16;
    return lds_read<uint16_t>(sb_at + P * 8 + row * 16);
  }
};

template <int H>
__device__ __forceinline__ f32x4 multiply(i32x4 b, int sb, i32x4 a, int sa, f32x4 acc) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4((i32x8){b[0], b[1], b[2], b[3], 0, 0, 0, 0},
                                                          (i32x8){a[0], a[1], a[2], a[3], 0, 0, 0, 0}, acc, 4, 4, H, sb,
                                                          H, sa);
}

// What a step finds read already: A's fragments of its first half, two of B's.
template <class T>
struct Ahead {
  i32x4 a[T::TM], b[2];
  int sa[T::TM], sb[2];
};

// Part 0 .. 3 of that, of a step of parity P.
template <class T, int P>
__device__ __forceinline__ void read_ahead(Ahead<T>& x, const Pass<T>& ps, int part) {
#pragma unroll
  for (int i = 0; i < T::TM; ++i)
    if (i % 4 == part) {
      x.a[i] = ps.template a_codes<0, P>(i);
      x.sa[i] = ps.template a_scales<P>(i);
    }
  if (part >= 2) {
    x.b[part - 2] = ps.template b_codes<0, P>(part - 2);
    x.sb[part - 2] = ps.template b_scales<P>(part - 2);
  }
}

// Stores of a pass a wave issues.
template <class T>
constexpr int stores(bool mx) {
  return T::TM * T::TN / (T::GATED ? 4 : 2) * (mx ? 2 : 1);
}

// One K step as 2 TN groups of TM products: half g / TN, column subtile g % TN.
// B's fragments are read two groups before their use and the last ones before
// group CUT.  A's part of the step's stage is read by group TM and given up at a
// barrier there (with few groups at CUT too), to be filled with step k, the one
// after the next (past the pass's last, a step of the next pass); B's part at
// CUT, where the next step's loads have arrived; the last four groups cover the
// reads of the next step's first fragments.  So a load has a step or more to
// arrive; and the loads are issued one a group, between products.  At the first
// step of a pass the stores of the pass before, issued after the loads that the
// step waits for, may still be on their way.
template <class T, int P, bool ACTIVE>
__device__ __forceinline__ void kstep(Pass<T>& ps, Ahead<T>& x, int k, bool first, bool mx, int wave) {
  constexpr int G = 2 * T::TN, CUT = G - 4;
  constexpr bool SPLIT = CUT > T::TM;
  constexpr int NEWER = SPLIT ? T::A_LOADS : 0;
  static_assert(!SPLIT || (T::A_LOADS <= CUT - T::TM && T::B_LOADS <= 4), "loads a group");
  i32x4 b[G], a1[T::TM];
  int sb[T::TN];
  b[0] = x.b[0];
  b[1] = x.b[1];
  sb[0] = x.sb[0];
  sb[1] = x.sb[1];
  int sa[T::TM];
#pragma unroll
  for (int i = 0; i < T::TM; ++i) sa[i] = x.sa[i];
  const auto read_b = [&](int g) {
    const int j = g % T::TN;
    if (g < T::TN) {
      b[g] = ps.template b_codes<0, P>(j);
      sb[j] = ps.template b_scales<P>(j);
    } else {
      b[g] = ps.template b_codes<1, P>(j);
    }
  };
  const auto group = [&](int g) {
    const int j = g % T::TN;
#pragma unroll
    for (int i = 0; i < T::TM; ++i) {
      if (g < T::TN)
        ps.acc[i][j] = multiply<0>(b[g], sb[j], x.a[i], sa[i], ps.acc[i][j]);
      else
        ps.acc[i][j] = multiply<1>(b[g], sb[j], a1[i], sa[i], ps.acc[i][j]);
    }
    // (an empty statement that names the sums: the products stay ahead of the
    // reads and loads that follow, instead of sinking past them with their
    // operands)
#pragma unroll
    for (int i = 0; i < T::TM; ++i) asm volatile("" : "+v"(ps.acc[i][j]));
    __builtin_amdgcn_sched_barrier(0);
  };
  const auto before_cut = [&](int g) {
    if (!ACTIVE) return;
    if (g < CUT - 2) {
      read_b(g + 2);
    } else {
      read_b(2 * g - CUT + 4);
      read_b(2 * g - CUT + 5);
    }
    // A's fragments of the second half, one a group
    if (g < T::TM) a1[g] = ps.template a_codes<1, P>(g);
    group(g);
  };
#pragma unroll
  for (int g = 0; g < T::TM; ++g) before_cut(g);
  if constexpr (SPLIT) {
    lds_barrier();
#pragma unroll
    for (int g = T::TM; g < CUT; ++g) {
      if (g - T::TM < T::A_LOADS) ps.template load_a<P>(g - T::TM, k, wave);
      before_cut(g);
    }
  }
  if (P == 0 && first) {
    if (mx)
      wait_vmem<NEWER + stores<T>(true)>();
    else
      wait_vmem<NEWER + stores<T>(false)>();
  } else {
    wait_vmem<NEWER>();
  }
  lds_barrier();
  if (P == 1) ps.flip_scales();
#pragma unroll
  for (int g = CUT; g < G; ++g) {
    if constexpr (!SPLIT) {
#pragma unroll
      for (int s = 0; s < T::A_LOADS; ++s)
        if (s % 4 == g - CUT) ps.template load_a<P>(s, k, wave);
    }
#pragma unroll
    for (int s = 0; s < T::B_LOADS; ++s)
      if (s % 4 == g - CUT) ps.template load_b<P>(s, k, wave);
    if (ACTIVE) {
      read_ahead<T, 1 - P>(x, ps, g - CUT);
      group(g);
    }
  }
  if (P == 0) ps.load_scales(k / 2, wave);
}

// Lane l's value of lane l ^ 8, in the lanes of `banks` (bit 2, 3: the upper
// eight of each 16); the others keep `mine`.
template <int BANKS>
__device__ __forceinline__ uint32_t from_half(uint32_t mine, uint32_t theirs) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)mine, (int)theirs, 0x128, 0xF, BANKS, false);  // row_ror:8
}

// The pass's rows of the sums, eight columns a lane and pair of subtiles.  Two
// pairs' BF16 results change places between the halves of 16 lanes, so that a
// store covers whole cache lines: eight rows of 64 columns, not 16 of 32.
// Every lane stores (through a buffer over the tile's rows; what is not to be
// stored, past its end), so that a wave's stores can be counted.
template <class T>
__device__ __forceinline__ void epilogue(const Pass<T>& ps, const MxGemmArgs& a, int row0, int col0, int wm, int wn, int lane,
                                         uint64_t rows_ok) {
  constexpr int STEP = T::GATED ? 4 : 2, PAIRS = T::TN / STEP;  // subtiles of 32 columns
  const int r = lane & 15, q = lane >> 4;
  const uint32_t rows = (uint32_t)min(T::BM, a.M - row0), N = (uint32_t)a.N;
  const bool mx = T::GATED && a.c_scale;
  const auto at = [](void* p, size_t bytes, uint32_t size) {
    return __builtin_amdgcn_make_buffer_rsrc(static_cast<uint8_t*>(p) + bytes, (short)0, (int)size, 0x00020000);
  };
  const __amdgpu_buffer_rsrc_t rc = at(a.C, (size_t)row0 * N * 2 / (mx ? 4 : 1), rows * N * 2 / (mx ? 4 : 1));
  const __amdgpu_buffer_rsrc_t rcs = at(a.c_scale, (size_t)row0 * N / 32, mx ? rows * N / 32 : 0u);
  // place of column n of the wave's row rl, or kSkip (below 2^28)
  const auto place = [&](int rl, uint32_t n) {
    return ((rows_ok >> rl) & 1) && n < N ? (uint32_t)(wm * T::WM + rl) * N + n : kSkip;
  };
  const uint32_t n0 = (uint32_t)(col0 + wn * PAIRS * 32);
#pragma unroll
  for (int i = 0; i < T::TM; ++i) {
    u32x4 out[PAIRS];
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) {
      const int j = p * STEP;
      float v[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const float x = ps.acc[i][j + t / 4][t % 4];
        if constexpr (T::GATED)
          v[t] = mx::gated(x, ps.acc[i][j + 2 + t / 4][t % 4]);
        else
          v[t] = x;
      }
      if (mx) {
        uint32_t top = mx::top8(v);
        top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
        const uint32_t code = mx::scale_code(top);
        const uint32_t word = code == 255u ? 0u : mx::codes8(v, mx::inverse(code));
        const uint32_t to = place(i * 16 + r, n0 + p * 32 + 8 * q);
        __builtin_amdgcn_raw_buffer_store_b32(word, rc, to == kSkip ? kSkip : to / 2, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b8((uint8_t)code, rcs, to == kSkip || q > 0 ? kSkip : to / 32, 0, 0);
      } else {
        const uint2 lo = pack_bf16x4(v[0], v[1], v[2], v[3]), hi = pack_bf16x4(v[4], v[5], v[6], v[7]);
        out[p] = (u32x4){lo.x, lo.y, hi.x, hi.y};
      }
    }
    if (mx) continue;
    if constexpr (PAIRS % 2 == 0) {
#pragma unroll
      for (int p = 0; p < PAIRS; p += 2) {
        u32x4 low, high;  // rows 0 .. 7 and 8 .. 15 of the 16
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          low[t] = from_half<0xC>(out[p][t], out[p + 1][t]);
          high[t] = from_half<0x3>(out[p + 1][t], out[p][t]);
        }
        const uint32_t n = n0 + p * 32 + (r >> 3) * 32 + 8 * q;
        const uint32_t t0 = place(i * 16 + (r & 7), n), t1 = place(i * 16 + 8 + (r & 7), n);
        __builtin_amdgcn_raw_buffer_store_b128(low, rc, t0 == kSkip ? kSkip : t0 * 2, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(high, rc, t1 == kSkip ? kSkip : t1 * 2, 0, 0);
      }
    } else {
#pragma unroll
      for (int p = 0; p < PAIRS; ++p) {
        const uint32_t to = place(i * 16 + r, n0 + p * 32 + 8 * q);
        __builtin_amdgcn_raw_buffer_store_b128(out[p], rc, to == kSkip ? kSkip : to * 2, 0, 0);
      }
    }
  }
}

// A pass: the tile's first row and column, the rows of the tile it may take, and
// the expert (-1: there is none).
struct Work {
  int row0, col0, lo, hi, e;
};

// The spans that the runs of one expert are cut into, as row0 << 8 | rows - 1: those of more than BM / 2 rows from the front of the list, the
// others from its back, both in the runs' order.
template <class T>
struct Spans {
  static constexpr int CAP = T::WG_PER_CU > 1 ? 1024 : 2048;
  uint32_t list[CAP];
  int heavy, light;  // how many; light < 0: not in runs

  // All threads call this; `scratch` is the stages.  Ends with a barrier.  More
  // runs than two for each expert and one are not taken (of rows in the experts'
  // order, each with padding behind its rows, there are as many): passes are
  // then at most that many more than full spans.
  __device__ __forceinline__ void build(uint8_t* scratch, const int32_t* ids, int M, int G) {
    constexpr int UNROLL = 8;
    const int words = (M + 63) / 64, lane = fresh_lane(), wave = (int)threadIdx.x >> 6;
    // a bit a row: does it begin a run?  Is it of no expert?
    uint64_t* first = reinterpret_cast<uint64_t*>(scratch);
    uint64_t* none = first + words;
    uint32_t* runs = reinterpret_cast<uint32_t*>(none + words);  // first row << 1 | of no expert
    light = -1;
    if (words * 16 + CAP * 4 > Lds<T>::BYTES) {
      __syncthreads();
      return;
    }
    const auto key = [&](int e) { return e < 0 || e >= G ? -1 : e; };
    for (int w0 = wave; w0 < words; w0 += T::WAVES * UNROLL) {
      int e[UNROLL], before[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int i = (w0 + u * T::WAVES) * 64 + lane;
        e[u] = i < M ? ids[i] : 0;
        before[u] = i < M && i > 0 ? ids[i - 1] : 0;
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int w = w0 + u * T::WAVES, i = w * 64 + lane;
        const uint64_t m = __ballot(i < M && (i == 0 || key(e[u]) != key(before[u])));
        const uint64_t z = __ballot(i < M && key(e[u]) < 0);
        if (lane == 0 && w < words) {
          first[w] = m;
          none[w] = z;
        }
      }
    }
    __syncthreads();
    if (wave == 0) {
      const auto prefix = [&](int v) {  // of the lanes before this one
        int x = v;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
          const int y = __shfl_up(x, d, 64);
          if (lane >= d) x += y;
        }
        return x - v;
      };
      const int most = min(2 * G + 1, CAP);
      int n = 0;
      for (int w0 = 0; w0 < words && n <= most; w0 += 64) {
        uint64_t m = w0 + lane < words ? first[w0 + lane] : 0;
        const uint64_t z = m ? none[w0 + lane] : 0;
        const int c = __popcll(m), p = prefix(c);
        for (int at = n + p; m && at < CAP; m &= m - 1, ++at) {
          const int b = __builtin_ctzll(m);
          runs[at] = (uint32_t)((w0 + lane) * 64 + b) << 1 | (uint32_t)(z >> b & 1);
        }
        n += __builtin_amdgcn_readlane(p + c, 63);
      }
      int full = 0, part = 0;
      bool fits = n <= most;
      for (int r0 = 0; r0 < n && fits; r0 += 64) {
        const int r = r0 + lane;
        const uint32_t run = r < n ? runs[r] : 1u;
        const int from = (int)(run >> 1), to = run & 1 ? from : r + 1 < n ? (int)(runs[r + 1] >> 1) : M;
        const int left = (to - from) % T::BM;
        const bool last_heavy = left > T::BM / 2;
        const int big = (to - from) / T::BM + last_heavy, small = left > 0 && !last_heavy;
        int at = full + prefix(big);
        const int back = part + prefix(small);
        full = __builtin_amdgcn_readlane(at + big, 63);
        part = __builtin_amdgcn_readlane(back + small, 63);
        fits = full + part <= CAP;
        if (!fits) break;
        for (int i = from; i < to - (small ? left : 0); i += T::BM) list[at++] = (uint32_t)i << 8 | (uint32_t)(min(to - i, T::BM) - 1);
        if (small) list[CAP - 1 - back] = (uint32_t)(to - left) << 8 | (uint32_t)(left - 1);
      }
      if (lane == 0) {
        heavy = full;
        light = fits ? part : -1;
      }
    }
    __syncthreads();
  }
};

// A workgroup's items.  Heavy tiles (windows with several experts, about two
// passes; spans of more than half their rows) come first in the order, and are
// taken to cost two light ones: whole rounds of heavy tiles, then one more heavy
// tile or two light ones a workgroup, then rounds of light ones.  With eight
// waves half the rows of a tile take one wave a SIMD, and little more than half
// the time.  So where the last round would leave half of the workgroups idle,
// each of its tiles goes to two of them, half of its rows each: of windows the
// light ones; of spans the heavy ones of the last round, where that is fewer
// rounds of light ones than going on as above.
struct Items {
  Items() = default;
  int tall, heavy;   // spans or windows, and heavy ones
  int total, heavies;  // tiles
  int rounds, rest, first, lights, halved;
  bool spans, split;  // split: the last heavy tiles are halved

  __device__ __forceinline__ Items(int tall_, int heavy_, int num_ntiles, bool halves, bool spans_)
      : tall(tall_), heavy(heavy_), total(tall_ * num_ntiles), heavies(heavy_ * num_ntiles), spans(spans_) {
    const int groups = (int)gridDim.x;
    rounds = heavies / groups;
    rest = heavies % groups;
    first = rest ? 2 * (groups - rest) : 0;
    lights = max(0, total - heavies - first);
    const int left = lights % groups;
    halved = halves && !spans && 2 * left <= groups ? left : 0;
    split = halves && spans && rest &&
            (2 * rest + total - heavies + groups - 1) / groups < 2 + (lights + groups - 1) / groups;
  }
  // Item n: the tile's place in the order and 0, or 1, 2 for its upper or lower
  // half; a place of -1 past the last.
  __device__ __forceinline__ int2 operator()(int n) const {
    const int groups = (int)gridDim.x, me = (int)blockIdx.x;
    if (n < rounds) return make_int2(n * groups + me, 0);
    n -= rounds;
    if (split) {
      const int i = n * groups + me;
      if (i < 2 * rest) return make_int2(rounds * groups + (i < rest ? i : i - rest), i < rest ? 1 : 2);
      return make_int2(heavies + i - 2 * rest < total ? heavies + i - 2 * rest : -1, 0);
    }
    if (rest) {
      if (me < rest) {
        if (n == 0) return make_int2(rounds * groups + me, 0);
        n -= 1;
      } else {
        if (n < 2) {
          const int i = heavies + n * (groups - rest) + (me - rest);
          return make_int2(i < total ? i : -1, 0);
        }
        n -= 2;
      }
    }
    const int i = n * groups + me, whole = lights - halved, i0 = heavies + first;
    if (i < whole) return make_int2(i0 + i, 0);
    if (i - whole < halved) return make_int2(i0 + i, 1);
    if (i - whole < 2 * halved) return make_int2(i0 + i - halved, 2);
    return make_int2(-1, 0);
  }
};

// The K loop of pass w, whose first two steps have arrived, and in its last two
// steps the first loads of the pass after it, whose operands `next_pass` sets.
// A wave without a row of the pass loads its part and computes nothing.
template <class T, bool ACTIVE, class Next>
__device__ __forceinline__ void k_loop(Pass<T>& ps, Ahead<T>& x, int nks, bool mx, int wave, Next next_pass) {
  for (int ks = 0; ks < nks; ks += 2) {
    int k = ks + 2;
    if (k == nks) {
      next_pass();
      k = 0;
    }
    kstep<T, 0, ACTIVE>(ps, x, k, ks == 0, mx, wave);
    kstep<T, 1, ACTIVE>(ps, x, k + 1, false, mx, wave);
  }
}

// A workgroup takes tiles gridDim.x apart, and their passes in turn; the loads
// go on from one pass to the next without a break.
template <class T>
__global__ __launch_bounds__(T::THREADS) void mx_tiles_kernel(const MxGemmArgs a, int num_windows, int num_ntiles) {
  constexpr int group_w = 4;  // rows of tiles that an XCD's tiles share (1 to 8: all within 3%)
  __shared__ __attribute__((aligned(1024))) uint8_t stages[Lds<T>::BYTES];
  __shared__ __attribute__((aligned(256))) int ids[3][T::BM];  // of the tile before, this one, and the next
  __shared__ union {
    Spans<T> spans;
    uint32_t windows[kPlanWords];
  } plan;
  __shared__ int plan_heavy;
  __shared__ Items items_lds;  // (not in registers over the K loop)

  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;
  Pass<T> ps;
  ps.init(a, stages, fresh_lane(), wave, wm, wn);
  const int nks = (ps.K128 + 3) / 4 * 2;  // an even number of steps
  const bool mx = T::GATED && a.c_scale;
  const auto clear = [&](int row, int col) __attribute__((always_inline)) {  // eight columns of a row of no expert
    const size_t to = (size_t)row * a.N + col;
    if (mx) {
      *reinterpret_cast<uint32_t*>(a.C + to / 2) = 0u;
      if (col % 32 == 0) a.c_scale[to / 32] = 0;
    } else {
      *reinterpret_cast<uint4*>(a.C + to * 2) = make_uint4(0, 0, 0, 0);
    }
  };

  if (a.m_indices) {
    // (rows gridDim.x apart, whose zeros this workgroup writes if they have no expert)
    int r = (int)(blockIdx.x + threadIdx.x * gridDim.x), e = r < a.M ? a.m_indices[r] : 0;
    plan.spans.build(stages, a.m_indices, a.M, a.G);
    const int light = __builtin_amdgcn_readfirstlane(plan.spans.light), spans = plan.spans.heavy;
    if (light >= 0) {
      if (threadIdx.x == 0) items_lds = Items(spans + light, spans, num_ntiles, T::WAVES == 8, true);
      for (;;) {
        const int lane = fresh_lane(), r0 = __builtin_amdgcn_readfirstlane(r);
        for (uint64_t none = __ballot(r < a.M && (e < 0 || e >= a.G)); none; none &= none - 1)
          for (int c = 8 * lane; c < a.N; c += 512) clear(r0 + __builtin_ctzll(none) * (int)gridDim.x, c);
        r += T::THREADS * (int)gridDim.x;
        if (__ballot(r < a.M) == 0) break;
        e = r < a.M ? a.m_indices[r] : 0;
      }
    } else {
      __syncthreads();
      build_plan<T::BM, T::THREADS>(plan.windows, &plan_heavy, a.m_indices, a.M, a.G, num_windows);
      if (threadIdx.x == 0) items_lds = Items(num_windows, plan_heavy, num_ntiles, T::WAVES == 8, false);
    }
  } else if (threadIdx.x == 0) {
    items_lds = Items(num_windows, 0, num_ntiles, T::WAVES == 8, false);
  }
  __syncthreads();

  // (inline at every call, so that what they change stays in registers)
  const auto items = [&](int n) __attribute__((always_inline)) {
    const int2 i = items_lds(n);
    return make_int2(__builtin_amdgcn_readfirstlane(i.x), __builtin_amdgcn_readfirstlane(i.y));
  };
  const auto in_spans = [&]() __attribute__((always_inline)) { return __builtin_amdgcn_readfirstlane((int)items_lds.spans) != 0; };
  const auto place_of = [&](int2 item) __attribute__((always_inline)) {
    int window, ntile;
    Work w{0, 0, 0, T::BM, -1};
    const int heavy = items_lds.heavy, tall = items_lds.tall;
    if (items_lds.spans) {
      const int split = heavy * num_ntiles;
      if (item.x < split) {
        map_tile(item.x, split, heavy, num_ntiles, group_w, window, ntile);
      } else {
        map_tile(item.x - split, (tall - heavy) * num_ntiles, tall - heavy, num_ntiles, group_w, window, ntile);
        window = Spans<T>::CAP - 1 - window;
      }
      const uint32_t span = plan.spans.list[window];
      w.row0 = (int)(span >> 8);
      w.hi = (int)(span & 255u) + 1;
    } else {
      plan_tile(plan.windows, heavy, item.x, num_windows, num_ntiles, group_w, window, ntile);
      w.row0 = window * T::BM;
    }
    w.col0 = ntile * T::COLS;
    if (item.y == 1) w.hi = min(w.hi, T::BM / 2);
    if (item.y == 2) w.lo = T::BM / 2;
    const auto same = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
    return Work{same(w.row0), same(w.col0), same(w.lo), same(w.hi), -1};
  };
  // The experts of an item's rows, read by direct loads an item ahead.
  const auto load_ids = [&](int2 item, int buf) __attribute__((always_inline)) {
    if (!a.m_indices || item.x < 0 || wave * 64 >= T::BM) return;
    const int row0 = place_of(item).row0;
    dma4(rsrc(a.m_indices + row0, (uint32_t)min(T::BM, a.M - row0) * 4u), lds_addr(&ids[buf][wave * 64]),
         (uint32_t)(wave * 64 + fresh_lane()) * 4u, 0);
  };
  const auto id_of = [&](int buf, const Work& w, int r) __attribute__((always_inline)) {
    if (w.row0 + r >= a.M || r < w.lo || r >= w.hi) return -2;  // never stored
    const int e = a.m_indices ? ids[buf][r] : 0;
    return e < 0 || e >= a.G ? -1 : e;
  };

  int item = 0, buf = 0;
  Work at{0, 0, 0, 0, -1};  // the item, and in it where the last pass was
  // The next pass: the next expert in the tile's window, in increasing order, or
  // the first of the next item that has one; e < 0 past the last.  The rows of
  // no expert of a new window are filled with zeros here, and the next item's
  // experts asked for.
  const auto enter = [&]() __attribute__((always_inline)) {
    const int lane = fresh_lane();
    at = place_of(items(item));
    if (!a.m_indices) return;
    load_ids(items(item + 1), buf == 2 ? 0 : buf + 1);
    if (in_spans()) return;
    for (int c = wave * 64 + lane; c < T::BM * (T::COLS / 8); c += T::THREADS) {
      const int r = c / (T::COLS / 8), col = at.col0 + c % (T::COLS / 8) * 8;
      if (id_of(buf, at, r) == -1 && col < a.N) clear(at.row0 + r, col);
    }
  };
  const auto advance = [&]() __attribute__((always_inline)) {
    const int lane = fresh_lane();
    for (bool moved = false;;) {
      int e = INT_MAX;
      if (!a.m_indices || in_spans()) {
        if (at.e < 0) e = a.m_indices ? __builtin_amdgcn_readfirstlane(ids[buf][at.lo]) : 0;
      } else {
#pragma unroll
        for (int r = 0; r < T::BM; r += 64) {
          const int v = id_of(buf, at, r + lane);
          if (v > at.e && v < e) e = v;
        }
        e = __builtin_amdgcn_readfirstlane(wave_min(e));
      }
      if (e != INT_MAX) {
        at.e = e;
        return;
      }
      at.e = -1;
      if (items(++item).x < 0) return;
      buf = buf == 2 ? 0 : buf + 1;
      if (moved) {  // the ids were asked for just now
        wait_vmem<0>();
        __syncthreads();
      }
      moved = true;
      enter();
    }
  };
  // Sets the loads' operands to those of pass n; past the last, to nothing.
  uint64_t rows_next = 0;  // the wave's rows of that pass
  const auto operands = [&](const Work& n) __attribute__((always_inline)) {
    const int lane = fresh_lane();
    const int none = n.e < 0 ? 1 : 0;
    uint64_t groups = 0;
    if (!none) {
#pragma unroll
      for (int r = 0; r < T::BM; r += 64) {  // eight rows a bit
        uint64_t m = __ballot(id_of(buf, n, r + lane) == n.e);
        if (r == wm * T::WM) rows_next = m;
        m |= m >> 1;
        m |= m >> 2;
        m |= m >> 4;
        m &= 0x0101010101010101ull;
        groups |= ((m * 0x0102040810204080ull) >> 56) << (r / 8);
      }
    } else {
      rows_next = 0;
    }
    ps.a_groups = groups;
    const Work z = none ? Work{0, 0, 0, 0, 0} : n;
    ps.ra = rsrc(a.A + (size_t)z.row0 * ps.Kp, (uint32_t)min(T::BM, a.M - z.row0) * ps.Kp);
    ps.set_expert(a, z.e, z.row0, z.col0, wave);
    if (none) {
      ps.ra[2] = ps.rs[2] = 0;
#pragma unroll
      for (int h = 0; h < ps.HALVES; ++h) ps.rb[h][2] = 0;
    }
  };

  if (items(0).x < 0) return;
  if (a.m_indices) {
    load_ids(items(0), 0);
    wait_vmem<0>();
    __syncthreads();
  }
  enter();
  if (a.m_indices) {
    wait_vmem<0>();
    __syncthreads();
  }
  advance();
  if (at.e < 0) return;
  operands(at);
#pragma unroll
  for (int i = 0; i < T::A_LOADS; ++i) ps.template load_a<0>(i, 0, wave);
#pragma unroll
  for (int i = 0; i < T::B_LOADS; ++i) ps.template load_b<0>(i, 0, wave);
  ps.load_scales(0, wave);
  ps.sc_next = T::SCALES;
#pragma unroll
  for (int i = 0; i < T::A_LOADS; ++i) ps.template load_a<1>(i, 1, wave);
#pragma unroll
  for (int i = 0; i < T::B_LOADS; ++i) ps.template load_b<1>(i, 1, wave);
  wait_vmem<0>();
  lds_barrier();
  Ahead<T> x;
  bool ahead = false;  // x holds the pass's first fragments
  for (;;) {
    const Work w = at;
    const uint64_t rows = rows_next;
    advance();
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
      for (int j = 0; j < T::TN; ++j) ps.acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    const auto next_pass = [&]() { operands(at); };
    if (rows != 0) {
      if (!ahead) {
#pragma unroll
        for (int part = 0; part < 4; ++part) read_ahead<T, 0>(x, ps, part);
      }
      k_loop<T, true>(ps, x, nks, mx, wave, next_pass);
      ahead = true;
    } else {
      k_loop<T, false>(ps, x, nks, mx, wave, next_pass);
      ahead = false;
    }
    // (opaque here, so that the stores' addresses are not kept over the K loop)
    int first_row = w.row0, first_col = w.col0;
    asm volatile("" : "+s"(first_row), "+s"(first_col));
    epilogue<T>(ps, a, first_row, first_col, wm, wn, fresh_lane(), rows);
    if (at.e < 0) break;
  }
  wait_vmem<0>();  // the loads past the last pass, which write zeros to LDS
}

template <class T>
hipError_t launch(const MxGemmArgs& a, hipStream_t s) {
  const int num_windows = (a.M + T::BM - 1) / T::BM, num_ntiles = (a.N + T::COLS - 1) / T::COLS;
  // (spans may be more than windows, by no more than the runs)
  const long long runs = a.m_indices ? std::min(2ll * a.G + 1, (long long)a.M) : 0;
  const long long total = (num_windows + runs) * num_ntiles;
  if (total > INT_MAX / 2) return hipErrorInvalidValue;
  const int grid = (int)std::min<long long>(total, (long long)a.num_cus * T::WG_PER_CU);
  hipLaunchKernelGGL(mx_tiles_kernel<T>, dim3((unsigned)grid), dim3(T::THREADS), 0, s, a, num_windows, num_ntiles);
  return hipGetLastError();
}

}  // namespace mx_tiles_detail

// Tiles of 256 rows x 256 columns, or of 128 x 128, two workgroups to a CU.
hipError_t launch_mx_tiles(const MxGemmArgs& a, bool large, hipStream_t s) {
  using namespace mx_tiles_detail;
  if (large) return a.gated ? launch<Cfg<256, 256, 4, 2, true>>(a, s) : launch<Cfg<256, 256, 4, 2, false>>(a, s);
  return a.gated ? launch<Cfg<128, 128, 2, 2, true>>(a, s) : launch<Cfg<128, 128, 2, 2, false>>(a, s);
}

hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t s) {
  const mx::Kernel k = mx::kernel_for(a.M, a.N, a.G, a.gated, a.num_cus);
  return k == mx::Kernel::kRows ? launch_mx_rows(a, s) : launch_mx_tiles(a, k == mx::Kernel::kLargeTiles, s);
}

}  // namespace fgg
