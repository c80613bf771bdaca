// prompt_attention: causal attention over whole prompts packed one after the
// other, grouped query heads.
//
//   o[t, h] = sum_{u <= t} p_u v_u / sum_{u <= t} p_u,
//   p_u = exp(scale q[t, h] . k[u] - m),  m = max_{u <= t} scale q[t, h] . k[u]
//
// over the tokens u of t's prompt.  A wave takes 32 queries of one head and goes
// once over the keys in blocks of 32 with the running maximum and sum.
// S^T = K Q^T on 32x32x16 MFMAs leaves a query's scores in one column of two
// lanes (l and l + 32); packed to BF16 they are the B operand of
// O^T = V^T P^T as they stand (contraction slot 8 h + 4 a + i of step s is
// token 16 s + 8 a + 4 h + i), with V^T read from LDS by transposed reads: the
// weights never leave their lane, and the two lanes of a query meet only when
// its maximum moves.  Scores, maxima, sums and outputs are FP32.  The weights are
// rounded to BF16, the matrix cores' input type; the sum that they are divided by
// is that of the rounded ones.  Against FP64 the result is off by 0.0018 to 0.0020
// of its size, 0.0016 of that the output's own rounding; as sums of two BF16
// values, which take the products with V twice, they add nothing to it, and 32
// heads of 128, prompts of 4096 and 8192 tokens, take 842 instead of 626 us, 24
// prompts of 17 to 1501 tokens on heads of 64 60 instead of 48.
//
// Four waves share the keys and values of a KV head through LDS, which direct
// loads fill 64 keys ahead.  Heads of 128 are bound by the matrix cores and the
// power they draw: 4 D operations a query and key.  Measured: 32 heads of 128,
// prompts of 4096 and 8192 tokens, 620 us, 1108 TFLOP/s, where a matrix product
// of 16384^3 reaches 1374; MFMAs busy 64% of the cycles, at a clock of 1.75 GHz;
// the same without loads or without softmax 566 us, without both 490 us.  Heads
// of 64 are bound by vector instructions: 55 plain ones and 16 exponentials (of
// four times the cycles) to 8 MFMAs a block; the same prompts 356 us, 965
// TFLOP/s; 24 prompts of 17 to 1501 tokens 49 us.
//
// A masked value must not reach the output even where it is infinite or NaN:
// masked scores are overwritten, but in the product with V a weight of 0
// times such a value is NaN.  Only in its last block does a wave have queries
// that do not see every key, so it looks that block's values over as it reads
// them; in the rare one that holds a value that is not finite, such values
// count as zeros in the product and are added by hand to the queries that
// see them.
#include "attn.h"
#include "attn_layout.h"

#include <type_traits>

namespace fgg {
namespace prompt_detail {

using namespace attn;

constexpr int kThreads = attn_layout::kThreads;
constexpr int kWaves = kThreads / 64;
// Queries of a workgroup whose waves take HP heads and are split KG ways over
// the keys.
constexpr int rows_of(int KG, int HP) { return 32 * kWaves / (KG * HP); }
constexpr float kSlack = 8.f;  // weights may reach 2^kSlack before a rescaling

// sum plus the product of two words' BF16 values.  (Words by value: of an
// element of a vector the compiler's bit cast takes the first one.)
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
constexpr uint32_t kOnes = 0x3F803F80u;
__device__ __forceinline__ float add_pair(uint32_t x, uint32_t y, float sum) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, x), __builtin_bit_cast(bf16x2, y), sum, false);
}

// Segment i of the packed tokens: 0 is what lies before the first prompt,
// 1 .. batch the prompts, batch + 1 what lies after the last.  It ends at the
// largest of the bounds up to its own (a bound that lies before an earlier one
// counts as that one), and there the next one begins: whatever the bounds hold,
// the segments share out the tokens [0, T], as the grid's size assumes.
__device__ __forceinline__ int bound(const PromptArgs& a, int i) {
  return i > a.batch ? a.T : min(max(a.starts[i], 0), a.T);
}
// Its tiles of `rows` queries.
__device__ __forceinline__ int row_tiles(int lo, int hi, int rows) { return (hi - lo + rows - 1) / rows; }

// A word's two BF16 values with zeros in the place of those that are infinite
// or NaN (an exponent of all ones plus one carries into the sign's bit).
__device__ __forceinline__ uint32_t without_odd(uint32_t w) {
  const uint32_t odd = (w & 0x7F807F80u) + 0x00800080u;
  return w & ~((odd & 0x8000u ? 0xFFFFu : 0u) | (odd & 0x80000000u ? 0xFFFF0000u : 0u));
}

// A direct load into LDS as lds_dma::dma16, except that the compiler may move
// LDS reads across it: what it overwrites is not read between two barriers.
__device__ __forceinline__ void dma16(i32x4 rs, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(voff),
               "s"(rs), "s"(soff)
               : "m0");
}

// Moves a buffer resource's base on.
__device__ __forceinline__ void advance(i32x4& rs, long long bytes) {
  const uint64_t at = ((uint64_t)(uint32_t)rs[1] << 32 | (uint32_t)rs[0]) + (uint64_t)bytes;
  rs[0] = (int)(uint32_t)at;
  rs[1] = (int)(uint32_t)(at >> 32);
}

// Sum and maximum of values that are not negative over a wave's lanes up to
// each: within rows of 16 lanes, then across them (DPP row_shr 1, 2, 4, 8,
// row_bcast 15, 31); and over the wave.
template <class Op>
__device__ __forceinline__ int wave_scan(int v, Op op) {
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true));
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true));
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true));
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true));
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));
  return v;
}
__device__ __forceinline__ int max_upto(int v) {
  return wave_scan(v, [](int x, int y) { return max(x, y); });
}
__device__ __forceinline__ int wave_sum(int v) {
  return __builtin_amdgcn_readlane(wave_scan(v, [](int x, int y) { return x + y; }), 63);
}
__device__ __forceinline__ int wave_max(int v) { return __builtin_amdgcn_readlane(max_upto(v), 63); }

// Maximum over a lane and its partner in the other half of the wave.
__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Registers and LDS are for two workgroups on a compute unit, with heads of 64
// for four: a short tile spends more time on its start and end than on its keys.
// (Bounds of three and four take the same time.)
template <int D, int KG, int HP>
__global__ __launch_bounds__(kThreads, D == 64 ? 4 : 2) void prompt_kernel(PromptArgs a) {
  static_assert(HP == 1 || KG == 1, "waves take several heads or several parts of the keys");
  constexpr int kRows = rows_of(KG, HP);
  constexpr int kGroups = kRows / 32;  // of 32 queries
  constexpr int kSteps = D / 16;    // k-steps of a QK product
  constexpr int kBlocks = D / 32;   // 32-row blocks of O^T
  constexpr int kRowBytes = D * 2;
  constexpr int kBlockBytes = 32 * kRowBytes;  // of a block of 32 keys
  constexpr int kChunks = D / 8;    // 16-byte chunks of a row
  constexpr int kLoads = kBlockBytes / 16 / kThreads;  // chunks of a block per thread
  // rings of four blocks of K and four of V: two are read while two land
  __shared__ __align__(16) uint8_t lds[8 * kBlockBytes];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int group = wave % kGroups, part = KG == 1 ? 0 : wave / kGroups;  // queries, keys

  // the row tile of this workgroup: heads fastest, so that the workgroups of
  // one KV head meet on the same XCDs' L2
  const int head_sets = a.q_heads / HP;
  const int hid = (int)blockIdx.x % head_sets, item = (int)blockIdx.x / head_sets;
  const int kvh = hid % a.kv_heads;
  const int head = kvh * (a.q_heads / a.kv_heads) + hid / a.kv_heads * HP + wave / kGroups % HP;
  // Each wave looks for it by itself.  Tiles with many keys come first.
  int seg, lo, hi, len, tile;
  const int segs = a.batch + 2;
  if (segs <= 64) {
    // over all prompts: level j holds the j-th tile of each segment with more
    // than j; highest levels first.  A segment to a lane.
    lo = max_upto(lane > 0 && lane < segs ? bound(a, lane - 1) : 0);
    hi = lane < segs ? max(lo, bound(a, lane)) : lo;
    const int n = row_tiles(lo, hi, kRows);
    auto from_level = [&](int j) { return wave_sum(max(n - j, 0)); };  // tiles at level j and above
    if (item >= from_level(0)) return;
    int below = 0, above = wave_max(n);  // from_level(below) > item >= from_level(above)
    int skip = 0;                        // from_level(above)
    while (above - below > 1) {
      const int mid = (above + below) >> 1;
      const int c = from_level(mid);
      if (c > item)
        below = mid;
      else
        above = mid, skip = c;
    }
    tile = below;
    // the (item - skip)-th segment that reaches this level
    const uint64_t reach = __ballot(n > tile);
    const int rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(reach >> 32),
                                               __builtin_amdgcn_mbcnt_lo((uint32_t)reach, 0));
    seg = __builtin_ctzll(__ballot(n > tile && rank == item - skip));
    lo = __builtin_amdgcn_readlane(lo, seg);
    hi = __builtin_amdgcn_readlane(hi, seg);
  } else {
    // prompt by prompt; several to a lane
    const int chunk = (segs + 63) / 64;
    const int i0 = min(lane * chunk, segs), i1 = min(i0 + chunk, segs);
    // tiles of the lane's segments if the first one begins at `from`, and the
    // last one's end
    auto tiles_from = [&](int from, int& end) {
      int sum = 0;
      end = from;
      for (int i = i0; i < i1; ++i) {
        const int to = max(end, bound(a, i));
        sum += row_tiles(end, to, kRows);
        end = to;
      }
      return sum;
    };
    int from = i0 > 0 ? bound(a, i0 - 1) : 0, end;
    int sum = tiles_from(from, end);
    const int earlier = __shfl_up(max_upto(end), 1, 64);
    if (lane > 0 && earlier > from) {  // only where bounds decrease
      from = earlier;
      sum = tiles_from(from, end);
    }
    int upto = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int x = __shfl_up(upto, off, 64);
      if (lane >= off) upto += x;
    }
    const uint64_t past = __ballot(item < upto);
    if (past == 0) return;
    const int src = __builtin_ctzll(past);
    int before = __builtin_amdgcn_readlane(upto - sum, src), n;
    lo = __builtin_amdgcn_readlane(from, src);
    for (seg = src * chunk;; ++seg) {
      hi = max(lo, bound(a, seg));
      n = row_tiles(lo, hi, kRows);
      if (item < before + n) break;
      before += n;
      lo = hi;
    }
    tile = n - 1 - (item - before);
  }
  seg = __builtin_amdgcn_readfirstlane(seg);
  lo = __builtin_amdgcn_readfirstlane(lo);
  len = __builtin_amdgcn_readfirstlane(hi) - lo;
  tile = __builtin_amdgcn_readfirstlane(tile);
  const int r0 = tile * kRows;
  const int w0 = r0 + group * 32;  // this wave's first query
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

    // Staging: a load of the four waves fills 256 chunks of a block (see the
    // layout's header).  Rows past the last key are not loaded and read as zeros.
    const int row_in = tid / kChunks;
    constexpr int kRowsPerLoad = kThreads / kChunks;
    const uint32_t k_at = attn_layout::stage_off(D, tid, false, a.k_token);
    const uint32_t v_at = attn_layout::stage_off(D, tid, true, a.v_token);
    const uint32_t k_load = (uint32_t)(kRowsPerLoad * 2) * (uint32_t)a.k_token;
    const uint32_t v_load = (uint32_t)(kRowsPerLoad * 2) * (uint32_t)a.v_token;
    const uint32_t lds0 = lds_dma::lds_addr(lds) + wave * 1024;
    auto stage = [&](const uint16_t* p, long long stride, uint32_t at, uint32_t load, int ring,
                     int block) __attribute__((always_inline)) {
      const int left = min(keys - block * 32, 32);
      const i32x4 rs = lds_dma::rsrc(p + (long long)block * 32 * stride,
                                     attn_layout::stage_bytes(D, left, stride));
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        dma16(rs, lds0 + (ring + (block & 3)) * kBlockBytes + i * (kThreads * 16),
              row_in + i * kRowsPerLoad < left ? at : lds_dma::kSkip, i * load);
    };
    auto stage_k = [&](int block) __attribute__((always_inline)) { stage(kp, a.k_token, k_at, k_load, 0, block); };
    auto stage_v = [&](int block) __attribute__((always_inline)) { stage(vp, a.v_token, v_at, v_load, 4, block); };
    // LDS addresses of the lane's K fragments in the first block of the ring
    typedef const __attribute__((address_space(3))) bf16x8* lds_bf16x8;
    uint32_t k_lds[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      k_lds[k] = lds_dma::lds_addr(lds) + part * kBlockBytes + attn_layout::k_read(D, lane, k);
      asm("" : "+v"(k_lds[k]));  // kept whole: a block's place is the read's constant offset
    }

    const int whole = r0 / 32;  // blocks that all queries of the workgroup see whole
    // The steps of a block of 32 keys: its scores, the largest one, the
    // weights, their product with the values.  `block` (a constant in the main
    // loop) is its place in the rings, less the wave's part of the keys.
    float mx;
    auto scores = [&](auto block, f32x16& s, auto between) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 16; ++j) s[j] = 0.f;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const bf16x8 kf = *(lds_bf16x8)(k_lds[k] + block * kBlockBytes);
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[k], s, 0, 0, 0);
        between(k);
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
      return x;
    };
    // The subtrahend follows the maximum only when that would let a weight
    // pass 2^kSlack: the outputs are then scaled down, which late blocks
    // almost never need.  So a lane looks at its own keys' scores, and only
    // then at those of the lane with the query's other keys.  A query's result
    // depends on its own scores only.
    auto follow = [&]() __attribute__((always_inline)) {
      if (__any((mx - m) * scale2 > kSlack)) {
        mx = half_max(mx);
        const bool grown = (mx - m) * scale2 > kSlack;
        const float alpha = grown ? __builtin_amdgcn_exp2f((m - mx) * scale2) : 1.f;
        m = grown ? mx : m;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) acc[i] *= alpha;
      }
    };
    // The sum is that of the weights as they multiply the values, rounded to
    // BF16: an instruction for two of them.
    auto weights = [&](const f32x16& s, bf16x8 (&pf)[2]) __attribute__((always_inline)) {
      const float ms = m == kNegInf ? 0.f : m * scale2;
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = __builtin_amdgcn_exp2f(fmaf(s[k * 8 + j], scale2, -ms));
        const u32x4 w = {pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]),
                         pack_bf16(p[6], p[7])};
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          sum0 = add_pair(w[j], kOnes, sum0);
          sum1 = add_pair(w[j + 1], kOnes, sum1);
        }
        pf[k] = __builtin_bit_cast(bf16x8, w);
      }
      l += sum0 + sum1;
    };
    auto add_odd = [&](int k0) __attribute__((always_inline)) {
      for (int u = k0; u <= query; ++u) {
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
    // V^T operand of 16 keys (half of a block) and 32 of its dims
    auto value = [&](auto block, int k, int i) __attribute__((always_inline)) {
      const uint8_t* vs = lds + (4 + part + block) * kBlockBytes;
      const u32x2 x[2] = {lds_read_tr(vs + attn_layout::v_read(D, lane, k, i, 0)),
                          lds_read_tr(vs + attn_layout::v_read(D, lane, k, i, 1))};
      return (u32x4){x[0][0], x[0][1], x[1][0], x[1][1]};
    };
    auto add_values = [&](auto block, const bf16x8 (&pf)[2]) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
          acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              __builtin_bit_cast(bf16x8, value(block, k, i)), pf[k], acc[i], 0, 0, 0);
    };
    // the same of the wave's last block
    auto add_last_values = [&](int block, const bf16x8 (&pf)[2]) __attribute__((always_inline)) {
      bool any = false;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        u32x4 v[kBlocks];
        float odd[2] = {0.f, 0.f};  // NaN, once a value is infinite or NaN (zero times it)
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          v[i] = value(block, k, i);
#pragma unroll
          for (int x = 0; x < 4; ++x) odd[x & 1] = add_pair(v[i][x], 0u, odd[x & 1]);
        }
        if (__any(odd[0] + odd[1] != 0.f)) {
          any = true;
#pragma unroll
          for (int i = 0; i < kBlocks; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) v[i][x] = without_odd(v[i][x]);
        }
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
          acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v[i]), pf[k],
                                                           acc[i], 0, 0, 0);
      }
      if (any && query < len) add_odd(w0);
    };
    // Takes the scores of a block through softmax and values while it computes
    // those of the wave's next one: matrix and vector work of one wave that do
    // not wait for each other.
    auto step = [&](auto block, auto block1, f32x16& s, f32x16& next, auto between) __attribute__((always_inline)) {
      follow();
      bf16x8 pf[2];
      scores(block1, next, between);
      weights(s, pf);
      add_values(block, pf);
      mx = largest(next);
    };
    // Landed after this at block u (even): V of blocks u and u + 1, and K of the
    // next ones, u + KG and u + KG + 1; every wave is done with the blocks
    // before those, whose places V of u + 2 and u + 3, K of u + KG + 2 and u +
    // KG + 3 take.
    auto turn = [&]() __attribute__((always_inline)) {
      lds_dma::wait_vmem<0>();
      lds_dma::lds_barrier();
    };
    auto stage_ahead = [&](int u) __attribute__((always_inline)) {
      stage_v(u + 2);
      stage_v(u + 3);
      stage_k(u + KG + 2);
      stage_k(u + KG + 3);
    };
    auto nothing = [](int) {};
    f32x16 s0, s1;
    // The bases move on by two blocks a turn, the rows of the loads are scalar
    // offsets, and the loads go out one at a time between matrix instructions.
    // Only near the last key is there something to check (`check`): rows past it
    // are not loaded and read as zeros.
    i32x4 k_rs = lds_dma::rsrc(kp + (KG + 2) * 32 * a.k_token, lds_dma::kSkip);
    i32x4 v_rs = lds_dma::rsrc(vp + 64 * a.v_token, lds_dma::kSkip);
    int v_left = keys - 64 - row_in, k_left = v_left - KG * 32;  // rows from this thread's to the last key
    auto load_v = [&](auto check, int block, int i) __attribute__((always_inline)) {
      dma16(v_rs, lds0 + (4 + (block + 2) % 4) * kBlockBytes + i * (kThreads * 16),
            check && i * kRowsPerLoad >= v_left ? lds_dma::kSkip : v_at, i * v_load);
    };
    auto load_k = [&](auto check, int block, int i) __attribute__((always_inline)) {
      dma16(k_rs, lds0 + (block + KG + 2 + i / kLoads) % 4 * kBlockBytes + i % kLoads * (kThreads * 16),
            check && i * kRowsPerLoad >= k_left ? lds_dma::kSkip : k_at, i * k_load);
    };
    auto main_turn = [&](auto check, auto block) __attribute__((always_inline)) {
      turn();
      if constexpr (KG == 1) {
        step(block, std::integral_constant<int, block + 1>{}, s0, s1, [&](int k) __attribute__((always_inline)) {
          if (k & 1) load_v(check, block, k >> 1);
        });
        step(std::integral_constant<int, block + 1>{}, std::integral_constant<int, (block + 2) % 4>{}, s1, s0,
             [&](int k) __attribute__((always_inline)) {
               if (k & 1) load_k(check, block, k >> 1);
             });
      } else {
        auto load = [&](int k) __attribute__((always_inline)) {
          if (k < 2 * kLoads)
            load_v(check, block, k);
          else
            load_k(check, block, k - 2 * kLoads);
        };
        step(block, std::integral_constant<int, (block + 2) % 4>{}, block == 0 ? s0 : s1, block == 0 ? s1 : s0, load);
      }
      advance(k_rs, 128 * a.k_token);
      advance(v_rs, 128 * a.v_token);
      if (check) {
        v_left -= 64;
        k_left -= 64;
      }
    };
    static_assert(kSteps == 4 * kLoads, "a load for each matrix instruction, or for each second one");
    stage_k(0);
    if (KG == 2) stage_k(1);
    stage_v(0);
    stage_v(1);
    stage_k(KG);
    stage_k(KG + 1);
    lds_dma::wait_vmem<4 * kLoads>();
    lds_dma::lds_barrier();
    scores(std::integral_constant<int, 0>{}, s0, nothing);
    mx = largest(s0);
    int u = 0;
    for (; u + KG + 6 <= whole; u += 4) {
      main_turn(std::false_type{}, std::integral_constant<int, 0>{});
      main_turn(std::false_type{}, std::integral_constant<int, 2>{});
    }
    v_left -= u * 32;
    k_left -= u * 32;
    for (; u + 4 <= whole; u += 4) {
      main_turn(std::true_type{}, std::integral_constant<int, 0>{});
      main_turn(std::true_type{}, std::integral_constant<int, 2>{});
    }
    int ring = 0;
    if (kGroups <= 2 && u + 2 <= whole) {
      turn();
      stage_ahead(u);
      if constexpr (KG == 1) {
        step(std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{}, s0, s1, nothing);
        step(std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{}, s1, s0, nothing);
      } else {
        step(std::integral_constant<int, 0>{}, std::integral_constant<int, 2>{}, s0, s1, nothing);
        s0 = s1;
      }
      u += 2;
      ring = 2;
    }
    // The diagonal: a group of queries sees as many of its blocks as groups come
    // before it, and a part of one more, its last.
    turn();
    bf16x8 pf[2];
    if constexpr (KG == 1) {
      if constexpr (kGroups <= 2) {
        if (kGroups == 1 ? u < whole : group > 0) {
          step(ring, ring + 1, s0, s1, nothing);
          s0 = s1;
          ++ring;
        }
      } else {
        stage_ahead(whole);
        if (group > 0) step(std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{}, s0, s1, nothing);
        if (group > 1) step(std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{}, s1, s0, nothing);
        if (keys > r0 + 64) turn();
        if (group > 2) step(std::integral_constant<int, 2>{}, std::integral_constant<int, 3>{}, s0, s1, nothing);
        if (group & 1) s0 = s1;
        ring = group;
      }
      hide(s0);
      mx = largest(s0);
      follow();
      weights(s0, pf);
      add_last_values(ring, pf);
    } else {
      if (part == group) {
        hide(s0);
        mx = largest(s0);
      }
      if (part <= group) {
        follow();
        weights(s0, pf);
        if (part == group)
          add_last_values(ring, pf);
        else
          add_values(ring, pf);
      }
    }
    lds_dma::wait_vmem<0>();  // no load may land in LDS after the wave's end
    if constexpr (KG == 2) {
      // the second part of the keys joins the first
      lds_dma::lds_barrier();
      float* to = reinterpret_cast<float*>(lds) + wave % 2 * ((kBlocks * 16 + 2) * 64) + lane;
      if (part) {
        to[0] = m;
        to[64] = l;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) to[(2 + i * 16 + j) * 64] = acc[i][j];
      }
      lds_dma::lds_barrier();
      if (part) return;
      const float m1 = fmaxf(m, to[0]);
      const float ms = m1 == kNegInf ? 0.f : m1;
      const float f0 = __builtin_amdgcn_exp2f((m - ms) * scale2);
      const float f1 = __builtin_amdgcn_exp2f((to[0] - ms) * scale2);
      l = l * f0 + to[64] * f1;
#pragma unroll
      for (int i = 0; i < kBlocks; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[i][j] = acc[i][j] * f0 + to[(2 + i * 16 + j) * 64] * f1;
    }
    l = xor_add(l, 32);
  } else if (part) {
    return;
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

// Workgroups of a launch: at most one partly filled tile a segment.
static long long grid_of(int T, int batch, int q_heads, int KG, int HP) {
  return ((long long)T / rows_of(KG, HP) + batch + 2) * (q_heads / HP);
}

template <int D, int KG, int HP>
hipError_t launch(const PromptArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)grid_of(a.T, a.batch, a.q_heads, KG, HP);  // (the host checks)
  hipLaunchKernelGGL((prompt_kernel<D, KG, HP>), dim3(grid), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

// Heads of one KV head that the waves of a workgroup take, where the keys are not
// split: as many of four as divide the group.  Fewer queries then make up the
// rows, and less is computed for nothing on the diagonal (24 prompts of 17 to
// 1501 tokens, D = 64, three sets of inputs in turn: 52 against 56 us with one head
// a workgroup; nothing gained on 8192 tokens, nor where the keys are split).
static int heads_together(int q_heads, int kv_heads) {
  const int group = q_heads / kv_heads;
  return group % 4 == 0 ? 4 : group % 2 == 0 ? 2 : 1;
}

long long prompt_workgroups(int T, int batch, int q_heads, int kv_heads) {
  return grid_of(T, batch, q_heads, 1, heads_together(q_heads, kv_heads));
}

template <int D>
hipError_t launch(const PromptArgs& a, hipStream_t s) {
  // A workgroup with 128 (head, query) rows loads a key for four waves.  Where
  // that would leave compute units without work or with one (long) item each,
  // halves of them, split over the keys, spread better: up to as many items as
  // compute units, or twice as many of heads of 64, four of which fit on one.
  // Measured, whole against split: 8 heads of 128, 4001 tokens 68 against 52 us, 32
  // of 1000 22.2 against 19.1 us, but 32 of 2048 46 against 49 us; 32 heads of 64,
  // 1500 tokens 21.8 against 18.3 us, 2048 30.7 against 28.5 us, 4096 86.9 against 86.1.
  // A split costs each workgroup a join and a larger tile per prompt, so
  // prompts have to be long for it, the longer the fuller the card is already (32
  // heads of 128, 20 prompts of 30 tokens 7.1 against 11.7 us, 4 of 200 10.1 against
  // 11.2 us, 2 of 400 12.8 against 12.4 us; 16 heads, 3 of 200 9.1 against 8.2 us; of
  // 64, 4 of 500 13.7 either way).
  const long long items = (long long)((a.T + 127) / 128) * a.q_heads;
  const bool split = items <= (D == 64 ? 2 : 1) * a.num_cus && items * 448 * a.batch <= (long long)a.num_cus * a.T;
  if (split) return launch<D, 2, 1>(a, s);
  switch (heads_together(a.q_heads, a.kv_heads)) {
    case 4: return launch<D, 1, 4>(a, s);
    case 2: return launch<D, 1, 2>(a, s);
    default: return launch<D, 1, 1>(a, s);
  }
}

hipError_t launch_prompt(const PromptArgs& a, hipStream_t s) {
  return a.D == 64 ? launch<64>(a, s) : launch<128>(a, s);
}

}  // namespace fgg
