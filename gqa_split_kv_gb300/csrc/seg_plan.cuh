// The partition of ragged work over a fixed grid.  Work comes in units (a sequence's KV
// head and 16 of its query rows, say) of whole tiles of 64 tokens; the tiles of all units
// stand in one line, and CTA c of n takes [c W / n, (c + 1) W / n) of its W tiles (n at most
// W, so that each has some).  So every CTA has the same number of tiles, whatever the lengths,
// and a unit
// is cut only where a CTA's range ends in it: its pieces are those of consecutive CTAs.  Piece (unit u,
// CTA c) has slot u + c of the partials: along the line u or c grows from one piece to the next, so no
// two share a slot, and units + n slots hold them all.
#pragma once

#include <cuda_runtime.h>

namespace da {

constexpr int kTile = 64;  // tokens
constexpr long long kMostTokens = 0x7fffffffLL - 1024;  // of a sequence: tiles and strides past the last fit 32 bits

// a / b of numbers that are not negative; most fit 32 bits, whose division is several times as fast.
__host__ __device__ __forceinline__ long long seg_div(long long a, long long b) {
  if (((unsigned long long)a | (unsigned long long)b) >> 32 == 0) return (unsigned)a / (unsigned)b;
  return a / b;
}
// CTAs of a grid that have tiles.
__host__ __device__ __forceinline__ int seg_used(long long W, int ctas) { return W < ctas ? (int)W : ctas; }
// First tile of CTA c.
__host__ __device__ __forceinline__ long long seg_start(long long W, int n, int c) { return seg_div(W * c, n); }
// The CTA that has tile x: the largest c with floor(c W / n) <= x.
__host__ __device__ __forceinline__ int seg_owner(long long W, int n, long long x) {
  return (int)seg_div((x + 1) * n - 1, W);
}

// Tiles of the tokens [base, min(len, cap)).
__host__ __device__ __forceinline__ int seg_tiles(int len, int cap, int base) {
  const int end = len < cap ? len : cap;
  return end > base ? (int)((unsigned)(end - base + kTile - 1) / kTile) : 0;
}

// Sums over the whole batch and over the sequences before b of their tiles; the warp
// executes it.  lens null: every sequence cap tokens.
struct SegSums {
  long long all, before;
};
__device__ __forceinline__ SegSums seg_sums(const int* lens, int B, int cap, int base, int b) {
  long long all = 0, before = 0;
  for (int i = threadIdx.x & 31; i < B; i += 32) {
    const int t = seg_tiles(lens ? lens[i] : cap, cap, base);
    all += t;
    if (i < b) before += t;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, d);
    before += __shfl_xor_sync(0xffffffffu, before, d);
  }
  return {all, before};
}

// The sequence whose per-sequence tiles (t_b each) hold position x of their line, x below
// the sum, and that line's start of it; the warp executes it.
struct SegAt {
  int b;
  long long start;
};
__device__ __forceinline__ SegAt seg_find(const int* lens, int B, int cap, int base, long long x) {
  const int lane = threadIdx.x & 31;
  long long at = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int i = b0 + lane;
    const long long t = i < B ? seg_tiles(lens ? lens[i] : cap, cap, base) : 0;
    long long s = t;  // inclusive sum over the lanes
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += o;
    }
    const unsigned holds = __ballot_sync(0xffffffffu, x < at + s);
    if (holds) {
      const int src = __ffs(holds) - 1;
      return {b0 + src, at + __shfl_sync(0xffffffffu, s - t, src)};
    }
    at += __shfl_sync(0xffffffffu, s, 31);
  }
  return {B, at};
}

}  // namespace da
