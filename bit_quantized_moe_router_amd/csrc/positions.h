// Positions of rows in an order by expert (or by adapter): tiles of them from
// the offsets alone, and the row of x that a position stands for.
#pragma once

#include "common.h"

namespace moe {

struct RowTile {
  int e, row, rows;  // expert, first position, positions (at most BT)
};

// Tile number `tile` of the order (expert, BT positions at a time), found by
// every wave from the offsets alone: lane l sums the tiles of E/64 consecutive
// experts, a scan over the lanes gives each its first tile.  Offsets are held
// inside [0, P] and made increasing, so that whatever they are no position
// outside the arrays is reached.  The loads do not wait for each other: this
// stands before everything else a small call does.
template <int BT>
__device__ __forceinline__ bool find_row_tile(const int32_t* __restrict__ offsets, int E, int P, int tile, RowTile* out) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) >> 6;  // at most 8
  const int e0 = lane * per;
  int off[9];
#pragma unroll
  for (int j = 0; j <= 8; j++)
    if (j <= per) off[j] = offsets[min(e0 + j, E)];  // past the last expert: no tiles
  int n[8], mine = 0;
#pragma unroll
  for (int j = 0; j < 8; j++) {
    n[j] = 0;
    if (j < per) {
      const int lo = min(max(off[j], 0), P), hi = min(max(off[j + 1], lo), P);
      n[j] = (hi - lo + BT - 1) / BT;
    }
    mine += n[j];
  }
  int end = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(end, d);
    if (lane >= d) end += v;
  }
  const int first = end - mine;
  const uint64_t hit = __ballot(tile >= first && tile < end);
  if (hit == 0) return false;
  const int owner = __builtin_ctzll(hit);
  int e = 0, row = 0, rows = 0, t = tile - first;
#pragma unroll
  for (int j = 0; j < 8; j++) {
    if (t >= 0 && t < n[j]) {
      const int lo = min(max(off[j], 0), P), hi = min(max(off[j + 1], lo), P);
      e = e0 + j;
      row = lo + t * BT;
      rows = min(hi - row, BT);
    }
    t -= n[j];
  }
  out->e = __builtin_amdgcn_readlane(e, owner);
  out->row = __builtin_amdgcn_readlane(row, owner);
  out->rows = __builtin_amdgcn_readlane(rows, owner);
  return true;
}

// r / d = (r * magic >> 32) >> shift for 0 <= r < 2^31, d >= 2.  With L = ceil(log2 d), shift = L - 1 and
// magic = floor(2^(31 + L) / d) + 1, so magic * d = 2^(31 + L) + e with 0 < e <= d: the quotient is off by
// r e / (d 2^(31 + L)) < 2^-L <= 1 / d, too little to reach the next whole number.
struct Divisor {
  uint32_t magic;
  int shift;
};

inline Divisor divisor(int d) {
  if (d < 2) return Divisor{0, 0};
  int log2 = 1;
  while ((1ll << log2) < d) log2++;
  return Divisor{(uint32_t)((1ull << (31 + log2)) / (uint32_t)d + 1), log2 - 1};
}

__device__ __forceinline__ int div_by(int r, Divisor d) { return (int)(__umulhi((uint32_t)r, d.magic) >> d.shift); }

}  // namespace moe
