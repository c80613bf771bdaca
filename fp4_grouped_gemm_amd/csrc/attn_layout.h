// LDS layout and staging offsets of prompt_attention's blocks of 32 keys, shared
// by the kernel (device) and a host check that enumerates every access
// (tests/attn_layout_check.cpp).  Plain integer arithmetic, no HIP types.
//
// A staged block holds 32 rows (keys or values of one head, D BF16 values);
// row r lies at r 2 D bytes, its 16-byte chunk c at chunk c ^ key(r), so that
// what one cycle of a fragment read touches lies in different banks (64 of 4
// bytes).  K: 16 bytes a lane, cycles of the 16 lanes with equal bit 5 and equal
// parity of bits 2..4, one chunk index of 16 rows that differ in their low four
// bits.  V (transposed reads): 8 bytes a lane, half a wave a cycle: 64 bytes
// of four consecutive rows.
#pragma once

#include "offsets.h"

namespace fgg {
namespace attn_layout {

constexpr int kThreads = 256;  // that stage a block together

FGG_HD int k_key(int D, int r) { return D == 128 ? r & 15 : (r >> 1) & 7; }
FGG_HD int v_key(int D, int r) {
  return D == 128 ? ((r & 3) << 2) | ((r >> 1) & 2) : ((r << 1) & 4) | ((r >> 1) & 2);
}

// Fragment of lane `lane` for contraction step k: row lane % 32, chunk 2 k +
// lane / 32.
FGG_HD int k_read(int D, int lane, int k) {
  const int r = lane & 31;
  return r * D * 2 + (((2 * k + (lane >> 5)) ^ k_key(D, r)) << 4);
}
// Transposed read e (of two) of lane `lane` for step k (16 rows) and block i of
// 32 dims: 8 bytes of row 16 k + 8 e + 4 (lane / 32) + lane % 16 / 4, dims 32 i
// + 16 (lane / 16 % 2) + 4 (lane % 4).
FGG_HD int v_read(int D, int lane, int k, int i, int e) {
  const int r = k * 16 + e * 8 + (lane >> 5) * 4 + ((lane & 15) >> 2);
  const int c = i * 4 + ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
  return r * D * 2 + ((c ^ v_key(D, r)) << 4) + (lane & 1) * 8;
}

// Staging: load j of thread t writes 16 bytes at (j kThreads + t) 16 of the
// block: row stage_row(j) + t / (D / 8), physical chunk t % (D / 8).  It fetches
// the chunk that belongs there at stage_off (the vector offset) plus
// stage_row(j) rows (the scalar one): a load moves a multiple of 16 rows, which
// leaves the keys as they are.
FGG_HD int stage_loads(int D) { return 32 * D * 2 / 16 / kThreads; }
FGG_HD int stage_rows(int D) { return kThreads / (D / 8); }  // of a load
FGG_HD uint32_t stage_off(int D, int t, bool value, long long stride) {
  const int r = t / (D / 8), c = t % (D / 8);
  return (uint32_t)(r * stride * 2) + (uint32_t)((c ^ (value ? v_key(D, r) : k_key(D, r))) << 4);
}
// Bytes from a block's first row that its `left` rows span.
FGG_HD uint32_t stage_bytes(int D, int left, long long stride) {
  return left > 0 ? ((uint32_t)(left - 1) * (uint32_t)stride + (uint32_t)D) * 2u : 0u;
}

}  // namespace attn_layout
}  // namespace fgg
