// paged_decode_attention: one new token a sequence against a paged cache.
//
//   o[h] = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q_h . k_t - m),
//   m = max_t scale q_h . k_t  over the cached tokens t of the sequence.
//
// One pass over the cache with the running maximum and sum; every key and
// value is read once for the (up to 16) query heads of its KV head, so the
// kernel is bound by HBM (2 r / bytes-per-value operations a byte for r
// heads).  Workgroups share the whole batch's work evenly: the tiles of 128
// tokens of all (sequence, KV head) rows in one list, a contiguous slice of
// it to each workgroup.  A workgroup finds its slice from the lengths
// itself, so nothing is read on the host and rows of any lengths balance.
// A row that lies in one slice is finished there; the pieces of the others
// are joined by a second kernel.  Measured: 64 sequences of 12000 to 32768
// tokens, 16 KV heads of 64, 804 us (5.4 GB, 6.8 TB/s; a kernel that only reads
// reaches 7.0), in E4M3 478 us (5.7 TB/s); 128 of 2000 to 8191, 8 KV heads of 128 in
// E4M3, 198 us (5.9 TB/s); 96 of 1 to 6000 66 us (4.7 TB/s); one of 130001 on 4 KV
// heads 52 us (5.1 TB/s), 6 of them the join.  Where a KV head has more than 16
// query heads its cache is read once for each 16 (64 sequences of 12000 to 32768
// tokens, one KV head of 128: 117 us with 16 query heads, 220 with 32).
//
// A wave takes 32 tokens of a tile.  S^T = K Q^T on 16x16x32 MFMAs: the A
// operand of lane l is row (token) l % 16, loaded from the cache straight
// into registers, and the result has the query head in lane % 16 and tokens
// 4 (l / 16) + i.  Those are, packed to BF16, the B operand of
// O^T = V^T P^T with contraction slot 8 (l / 16) + 4 a + i for token
// 16 a + 4 (l / 16) + i: P never leaves its lane.  The A operand V^T comes
// from LDS by transposed reads of 4 tokens each.  The matrix cores take BF16,
// so a weight goes in as the sum of two BF16 values, 16 bits in all: the
// second product costs next to nothing under the memory's time (197.4 against
// 196.2 us for 128 sequences of 2000 to 8191 tokens in E4M3, nothing in BF16) and
// takes the weights' rounding out of the result.  Scores, maxima, sums and
// outputs are FP32.  (A weight below 2^-110 has a second half of 0: times an
// infinite value that is NaN, where the first half gives infinity.)
#include "attn.h"
#include "attn_list.h"

namespace fgg {
namespace decode_detail {

using namespace attn;

using attn_list::kTile;
using attn_list::kWaveTokens;
using attn_list::tiles_of;

constexpr int kMaxHeads = 16;  // query heads of a KV head in one row of work

// Waves of a workgroup, and workgroups on a compute unit.  Registers allow
// three waves a SIMD: three workgroups of four waves that share the list, or
// one of twelve that takes a whole row.  The latter needs no join and no second
// launch; its waves take 384 tokens at once.  It is taken for tables of one such
// step (one sequence of 300 tokens, 8 KV heads: 7.2 against 8.8 us), of two where
// the rows fill half of the card (240 rows of 700 tokens 18.4 against 23.5 us, 128
// rows 16.0 against 15.8; one sequence of 517 tokens 9.3 against 8.9, of 700 11.1
// against 8.9 us), and of four where they fill it (256 rows of 1000 tokens 23.6
// against 29.0 us, 1024 rows 90.6 against 91.1 us).
constexpr int kListWaves = attn_list::kWaves, kListPerCu = 3;
constexpr int kWholeWaves = 12;
constexpr int kWholeStep = kWholeWaves * kWaveTokens;

__device__ __forceinline__ int length_of(const DecodeArgs& a, int b) {
  const long long cap = (long long)a.c.width << a.c.page_shift;
  const int n = a.lengths[b];
  return n < 0 ? 0 : n > cap ? (int)cap : n;
}
// Rows of work of a KV head: its query heads by kMaxHeads.
__device__ __forceinline__ int head_groups(const DecodeArgs& a) {
  return (a.q_heads / a.c.kv_heads + kMaxHeads - 1) / kMaxHeads;
}

// The join has a place for each row of the batch if there are no more rows
// than slices, else one for each slice (a slice holds the beginning of one
// shared row at most).
__device__ __host__ __forceinline__ bool joins_by_row(int rows, int workgroups) {
  return rows <= workgroups;
}

// A load of what this launch does not read again.  Keys and values of a batch
// are far more than the caches hold, and a load that does not displace what
// they hold reads faster: 64 sequences of 12000 to 32768 tokens 804 against 891
// us (6.8 against 6.1 TB/s), 128 of 2000 to 8191 in E4M3 198 against 220, 96 of 1 to
// 6000 66 against 73 us.
__device__ __forceinline__ u32x4 once(const uint8_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}

// kWhole: one row a workgroup, nothing to join.  Else a slice of the list.
template <int D, bool FP8, int kWaves, bool kWhole>
__global__ __launch_bounds__(kWaves * 64, kWhole ? kWaves / 4 : kListPerCu) void decode_kernel(DecodeArgs a) {
  constexpr int kThreads = kWaves * 64;
  constexpr int kStep = kWaves * kWaveTokens;   // tokens that the waves take at once
  constexpr int kSteps = D / 32;                // k-steps of a QK product
  constexpr int kBlocks = D / 16;               // 16-row blocks of O^T
  constexpr int kRow = D * 2 + 32;              // LDS bytes of a staged V row (BF16)
  constexpr int kVB = FP8 ? D : D * 2;          // bytes of a cached row
  constexpr int kLoads = kWaveTokens * kVB / 16 / 64;  // 16-byte pieces of 32 rows per lane
  constexpr int kLanesPerRow = kVB / 16;
  constexpr int kOutRow = D + 4;                // floats of a row in the join's LDS
  constexpr int kStageBytes = kWaves * kWaveTokens * kRow;
  constexpr int kJoinBytes = kWaves * kMaxHeads * kOutRow * 4;
  __shared__ __align__(16) uint8_t stage[kStageBytes > kJoinBytes ? kStageBytes : kJoinBytes];
  __shared__ float ml[kWaves][kMaxHeads][2];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int groups = head_groups(a);
  const int group_heads = a.q_heads / a.c.kv_heads;
  const int rows = a.c.kv_heads * groups;  // rows of work of a sequence

  // This workgroup's slice of the list, and the sequence that it begins in.
  // Each wave goes over the lengths by itself, some to a lane.
  int b, before, total, pos, end;  // `before`: tiles of one row of each earlier sequence
  bool by_row = false;
  if constexpr (kWhole) {
    b = (int)blockIdx.x / rows;
    before = total = 0;
    pos = (int)blockIdx.x - b * rows;  // the row
    end = pos + 1;
  } else {
    const int chunk = (a.c.batch + 63) / 64;
    const int b0 = lane * chunk, b1 = min(b0 + chunk, a.c.batch);
    int sum = 0;
    for (int i = b0; i < b1; ++i) sum += tiles_of(length_of(a, i));
    int upto = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int u = __shfl_up(upto, off, 64);
      if (lane >= off) upto += u;
    }
    total = __builtin_amdgcn_readlane(upto, 63) * rows;
    pos = attn_list::slice_start(blockIdx.x, total, gridDim.x);
    const int first = min(pos, total - 1);
    // the lane whose sequences hold tile `first`, then the sequence
    const int src = __builtin_ctzll(__ballot(first < upto * rows));
    before = __builtin_amdgcn_readlane(upto - sum, src);
    for (b = src * chunk;; ++b) {
      const int n = tiles_of(length_of(a, b));
      if (first < (before + n) * rows) break;
      before += n;
    }
    end = attn_list::slice_start(blockIdx.x + 1, total, gridDim.x);
    by_row = joins_by_row(a.c.batch * rows, (int)gridDim.x);
    if (!by_row && tid == 0) a.split[blockIdx.x].first = -1;
  }

  uint8_t* const my_stage = stage + wave * (kWaveTokens * kRow);
  while (pos < end) {
    const int len = length_of(a, b);
    const int n = kWhole ? (len + kStep - 1) / kStep : tiles_of(len);
    const int rel = pos - before * rows;
    const int row = kWhole ? pos : rel / n, t0 = kWhole ? 0 : rel - row * n;
    const int t1 = kWhole ? n : min(n, t0 + end - pos);
    const int kvh = row / groups, g0 = (row - kvh * groups) * kMaxHeads;
    const int heads = min(kMaxHeads, group_heads - g0);
    const int head0 = kvh * group_heads + g0;

    // Q^T operand: head `col`; the dims of step s, slot 8 quad + j are the
    // ones that this lane's 16-byte pieces of K hold
    bf16x8 qf[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int d = FP8 ? (s >> 1) * 64 + quad * 16 + (s & 1) * 8 : s * 32 + quad * 8;
      u32x4 w = {0, 0, 0, 0};
      if (col < heads)
        w = *reinterpret_cast<const u32x4*>(a.q + b * a.q_seq + (head0 + col) * a.q_head + d);
      qf[s] = __builtin_bit_cast(bf16x8, w);
    }
    const float kscale = FP8 && a.c.k_scale ? a.c.k_scale[kvh] : 1.0f;
    const float scale2 = a.scale * kscale * kLog2e;
    const int32_t* table = a.c.table + b * a.c.table_stride;
    const uint8_t* kbase = a.c.k + kvh * a.c.k_head;
    const uint8_t* vbase = a.c.v + kvh * a.c.v_head;

    f32x4 acc[kBlocks];
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) acc[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
    float m = kNegInf, l = 0.f;

    for (int t = t0; t < t1; ++t) {
      const int tok0 = attn_list::first_token(t, kStep, wave);
      if (tok0 >= len) break;
      // lane L looks up token tok0 + L % 32: its page, or -1
      const int tok = tok0 + (lane & 31);
      int page = -1;
      if (tok < len) {
        page = table[tok >> a.c.page_shift];
        if (page >= a.c.num_pages) page = -1;
      }
      const uint32_t valid = (uint32_t)__ballot(page >= 0);
      if (valid == 0) continue;
      // a token without a page reads page 0 and is masked below
      const int safe = page < 0 ? 0 : page;
      const int slot = tok & ((1 << a.c.page_shift) - 1);
      u32x4 kw[2][kSteps * (FP8 ? 1 : 2) / 2], vw[kLoads];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int src = g * 16 + col;
        const int pg = __shfl(safe, src, 64), sl = __shfl(slot, src, 64);
        const uint8_t* p = kbase + pg * a.c.k_page + sl * a.c.k_token + quad * 16;
#pragma unroll
        for (int s = 0; s < kVB / 64; ++s) kw[g][s] = once(p + s * 64);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int src = i * (64 / kLanesPerRow) + lane / kLanesPerRow;
        const int pg = __shfl(safe, src, 64), sl = __shfl(slot, src, 64);
        vw[i] = once(vbase + pg * a.c.v_page + sl * a.c.v_token + (lane % kLanesPerRow) * 16);
      }
      // scores
      float s[8];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          bf16x8 kf;
          if constexpr (FP8) {
            const u32x4 w = kw[g][k >> 1];
            kf = __builtin_bit_cast(bf16x8, fp8x8_to_bf16((u32x2){w[(k & 1) * 2], w[(k & 1) * 2 + 1]}));
          } else {
            kf = __builtin_bit_cast(bf16x8, kw[g][k]);
          }
          c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[k], c, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[g * 4 + i] = c[i] * scale2;
      }
      if (valid != 0xFFFFFFFFu) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!((valid >> ((i >> 2) * 16 + quad * 4 + (i & 3))) & 1)) s[i] = kNegInf;
        // what the cache holds there may be NaN, and 0 x NaN is not 0
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          if (!((valid >> (i * (64 / kLanesPerRow) + lane / kLanesPerRow)) & 1))
            vw[i] = (u32x4){0, 0, 0, 0};
      }
      float mx = s[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s[i]);
      mx = xor_max(xor_max(mx, 16), 32);
      const float m1 = fmaxf(m, mx);
      const float ms = m1 == kNegInf ? 0.f : m1;
      const float alpha = __builtin_amdgcn_exp2f(m - ms);
      m = m1;
      float p[8], sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = __builtin_amdgcn_exp2f(s[i] - ms);
        sum += p[i];
      }
      l = l * alpha + sum;  // of this lane's tokens; the quads are added at the end
      // Each weight as the sum of two BF16 values: its upper half, and what is
      // left plus 2^-23 of it, which keeps the second one above zero (0 times
      // an infinite value would be NaN).
      u32x4 ph, pl;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = __float_as_uint(p[2 * i]), y = __float_as_uint(p[2 * i + 1]);
        ph[i] = __builtin_amdgcn_perm(y, x, 0x07060302u);
        pl[i] = pack_bf16(fmaf(p[2 * i], 1.f + 0x1p-23f, -__uint_as_float(x & 0xFFFF0000u)),
                          fmaf(p[2 * i + 1], 1.f + 0x1p-23f, -__uint_as_float(y & 0xFFFF0000u)));
      }
      // values through LDS (rows of BF16)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = i * (64 / kLanesPerRow) + lane / kLanesPerRow;
        uint8_t* dst = my_stage + r * kRow + (lane % kLanesPerRow) * (FP8 ? 32 : 16);
        if constexpr (FP8) {
          *reinterpret_cast<u32x4*>(dst) = fp8x8_to_bf16((u32x2){vw[i][0], vw[i][1]});
          *reinterpret_cast<u32x4*>(dst + 16) = fp8x8_to_bf16((u32x2){vw[i][2], vw[i][3]});
        } else {
          *reinterpret_cast<u32x4*>(dst) = vw[i];
        }
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) {
        const uint8_t* src = my_stage + (quad * 4 + (col >> 2)) * kRow + i * 32 + (col & 3) * 8;
        const u32x2 lo = lds_read_tr(src), hi = lds_read_tr(src + 16 * kRow);
        const bf16x8 vf = __builtin_bit_cast(bf16x8, (u32x4){lo[0], lo[1], hi[0], hi[1]});
        acc[i] *= alpha;
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, __builtin_bit_cast(bf16x8, ph), acc[i], 0, 0, 0);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, __builtin_bit_cast(bf16x8, pl), acc[i], 0, 0, 0);
      }
      __builtin_amdgcn_wave_barrier();
    }
    l = xor_add(xor_add(l, 16), 32);

    // join the waves
    __syncthreads();
    float* ow = reinterpret_cast<float*>(stage) + (wave * kMaxHeads + col) * kOutRow;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) *reinterpret_cast<f32x4*>(ow + i * 16 + quad * 4) = acc[i];
    if (quad == 0) {
      ml[wave][col][0] = m;
      ml[wave][col][1] = l;
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == n;
    if (!kWhole && t0 == 0 && tid == 0) {
      if (!whole)
        a.split[by_row ? b * rows + row : (int)blockIdx.x] =
            SplitRow{(int)blockIdx.x, attn_list::slice_of(pos + n - 1, total, gridDim.x), b, head0, heads, {}};
      else if (by_row)
        a.split[b * rows + row].first = -1;
    }
    const int piece = (int)blockIdx.x * 2 + (t0 > 0 ? 0 : 1);
    for (int x = tid; x < heads * (D / 4); x += kThreads) {
      const int h = x / (D / 4), d = x % (D / 4) * 4;
      float M = kNegInf;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) M = fmaxf(M, ml[w][h][0]);
      const float Ms = M == kNegInf ? 0.f : M;
      float L = 0.f;
      f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(ml[w][h][0] - Ms);
        L += f * ml[w][h][1];
        o += f * *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(stage) +
                                                 (w * kMaxHeads + h) * kOutRow + d);
      }
      if (whole) {
        const float vs = FP8 && a.c.v_scale ? a.c.v_scale[kvh] : 1.0f;
        o *= L == 0.f ? 0.f : vs / L;
        *reinterpret_cast<uint2*>(a.out + ((long long)b * a.q_heads + head0 + h) * D + d) =
            pack_bf16x4(o[0], o[1], o[2], o[3]);
      } else {
        *reinterpret_cast<f32x4*>(a.part_o + ((long long)piece * kMaxHeads + h) * D + d) = o;
        if (d == 0)
          *reinterpret_cast<f32x2*>(a.part_ml + (piece * kMaxHeads + h) * 2) = (f32x2){M, L};
      }
    }
    if constexpr (kWhole) return;
    __syncthreads();  // the stage is free again
    pos += t1 - t0;
    if (t1 == n && row == rows - 1) {
      before += n;
      ++b;
    }
  }
}

// Joins the pieces of the rows that the slices of several workgroups share:
// kWide waves to a head of the row in place x, if there is one.  The pieces
// of a head go to groups of D / 4 lanes in turn, kAhead of them loaded at
// once, so that four waves take the most there can be, a row over all slices,
// in few round trips to memory.
constexpr int kAhead = 8;
constexpr int kJoinWaves = 4;

template <int D, int kWide>
__global__ __launch_bounds__(kJoinWaves * 64) void join_kernel(DecodeArgs a) {
  constexpr int kLanes = D / 4, kSets = kWide * 64 / kLanes, kHeads = kJoinWaves / kWide;
  __shared__ __align__(16) float red_o[kHeads][kSets][D];
  __shared__ float red_ml[kHeads][kSets][2];
  const SplitRow row = a.split[blockIdx.x];
  const int first = row.first, last = row.last;
  if (first < 0) return;
  const int which = threadIdx.x / (kWide * 64), t = threadIdx.x % (kWide * 64);
  const int h = min((int)blockIdx.y * kHeads + which, kMaxHeads - 1);
  const int set = t / kLanes, d = (t % kLanes) * 4;
  float m = kNegInf, l = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  for (int w0 = first + set; w0 <= last; w0 += kSets * kAhead) {
    f32x2 ml[kAhead];
    f32x4 x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      // past the last piece: the last one again, without weight
      const int w = min(w0 + i * kSets, last);
      const int p = (w * 2 + (w == first ? 1 : 0)) * kMaxHeads + h;
      ml[i] = *reinterpret_cast<const f32x2*>(a.part_ml + p * 2);
      x[i] = *reinterpret_cast<const f32x4*>(a.part_o + (long long)p * D + d);
    }
    float m1 = m;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) m1 = fmaxf(m1, ml[i][0]);
    const float ms = m1 == kNegInf ? 0.f : m1;
    const float alpha = __builtin_amdgcn_exp2f(m - ms);
    m = m1;
    l *= alpha;
    o *= alpha;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (w0 + i * kSets > last) continue;
      const float f = __builtin_amdgcn_exp2f(ml[i][0] - ms);
      l += f * ml[i][1];
      o += f * x[i];
    }
  }
  *reinterpret_cast<f32x4*>(&red_o[which][set][d]) = o;
  if (d == 0) {
    red_ml[which][set][0] = m;
    red_ml[which][set][1] = l;
  }
  __syncthreads();
  if (t >= kLanes || (int)blockIdx.y * kHeads + which >= row.heads) return;
  float M = kNegInf;
#pragma unroll
  for (int i = 0; i < kSets; ++i) M = fmaxf(M, red_ml[which][i][0]);
  const float ms = M == kNegInf ? 0.f : M;
  float L = 0.f;
  f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kSets; ++i) {
    const float f = __builtin_amdgcn_exp2f(red_ml[which][i][0] - ms);
    L += f * red_ml[which][i][1];
    r += f * *reinterpret_cast<const f32x4*>(&red_o[which][i][d]);
  }
  const int head = row.head0 + h;
  const float vs =
      a.c.fp8 && a.c.v_scale ? a.c.v_scale[head / (a.q_heads / a.c.kv_heads)] : 1.0f;
  r *= L == 0.f ? 0.f : vs / L;
  *reinterpret_cast<uint2*>(a.out + ((long long)row.b * a.q_heads + head) * D + d) =
      pack_bf16x4(r[0], r[1], r[2], r[3]);
}

// Rows of work of a batch.
long long rows_of(int batch, int q_heads, int kv_heads) {
  return (long long)batch * kv_heads * ((q_heads / kv_heads + kMaxHeads - 1) / kMaxHeads);
}

template <int D, bool FP8>
hipError_t launch(const DecodeArgs& a, int workgroups, hipStream_t s) {
  const long long rows = rows_of(a.c.batch, a.q_heads, a.c.kv_heads);
  if (workgroups == 0) {
    hipLaunchKernelGGL((decode_kernel<D, FP8, kWholeWaves, true>), dim3((unsigned)rows),
                       dim3(kWholeWaves * 64), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((decode_kernel<D, FP8, kListWaves, false>), dim3(workgroups),
                     dim3(kListWaves * 64), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int heads = a.q_heads / a.c.kv_heads < kMaxHeads ? a.q_heads / a.c.kv_heads : kMaxHeads;
  // Where there are fewer rows than slices, rows have many pieces.
  if (joins_by_row((int)rows, workgroups))
    hipLaunchKernelGGL((join_kernel<D, kJoinWaves>), dim3((unsigned)rows, heads),
                       dim3(kJoinWaves * 64), 0, s, a);
  else
    hipLaunchKernelGGL((join_kernel<D, 1>), dim3(workgroups, (heads + kJoinWaves - 1) / kJoinWaves),
                       dim3(kJoinWaves * 64), 0, s, a);
  return hipGetLastError();
}

}  // namespace decode_detail

using namespace decode_detail;

int decode_workgroups(int batch, int q_heads, int kv_heads, long long max_len, int num_cus) {
  const long long rows = rows_of(batch, q_heads, kv_heads);
  const int steps = rows >= num_cus ? 4 : 2 * rows >= num_cus ? 2 : 1;
  // (a launch takes fewer than 2^32 threads)
  if (max_len <= steps * kWholeStep && rows * (kWholeWaves * 64) <= 0xFFFFFFFFLL) return 0;
  const long long tiles = rows * ((max_len + kTile - 1) / kTile);
  const long long cap = (long long)kListPerCu * num_cus;
  return (int)(tiles < cap ? tiles : cap);
}

size_t decode_workspace(int workgroups, int D) {
  return (size_t)workgroups * (2 * kMaxHeads * (D + 2) * sizeof(float) + sizeof(SplitRow));
}

hipError_t launch_decode(const DecodeArgs& a, int workgroups, hipStream_t s) {
  if (a.D == 64)
    return a.c.fp8 ? launch<64, true>(a, workgroups, s) : launch<64, false>(a, workgroups, s);
  return a.c.fp8 ? launch<128, true>(a, workgroups, s) : launch<128, false>(a, workgroups, s);
}

}  // namespace fgg
