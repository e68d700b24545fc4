// Cutting caches down to the tokens of the largest weights.
//   select    per (sequence, KV head): the kept positions in ascending order;
//   move      the rows, scales and weights of those positions to 0, 1, ...
#pragma once

#include <cstdint>

#include "device_error.cuh"
#include "ptx.cuh"
#include "weights_kernel.cuh"

namespace da {

struct EvictParams {
  void *k, *v;  // rows of `row_bytes` a token and head
  float *ks, *vs, *weights;
  const int *page_table, *seq_lens;
  int *kept, *new_lens;
  void *k_out, *v_out;  // the cache's own where it is compacted in place
  float *ks_out, *vs_out, *weights_out;
  int B, Hkv, cap, slab;  // slab: rows a sequence, or a page
  int max_pages, num_pages;
  int keep, first, recent;
  int row_bytes;
  int in_place, out_ctx;
  int parts;    // CTAs that share a (sequence, head, tensor)'s rows (in place: 1)
  int columns;  // CTAs that share its rows' bytes
};

constexpr int kEvictThreads = 1024;

// The need-th largest of the candidates' keys is found 11, 11 and 10 bits at a time, by counting
// the keys of each digit in shared memory (zeros, of which there may be very many, are counted
// in registers); then every warp counts its own stretch of positions and, after one sum over
// the warps, writes its kept ones in place.  The weights are read five times, from L1 but for
// the first.
template <bool PAGED>
__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int hist[2048];
  __shared__ int s_warp[32], s_warp_eq[32], s_zero, s_digit, s_above;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int b = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
  const int L = seg_len(p.seq_lens, b, p.cap);
  int* kept = p.kept + (size_t)blockIdx.x * p.keep;
  if (h == 0 && threadIdx.x == 0) p.new_lens[b] = min(L, p.keep);
  if (L <= p.keep) {
    for (int i = threadIdx.x; i < p.keep; i += kEvictThreads) kept[i] = i < L ? i : -1;
    return;
  }
  const int lo = p.first, hi = L - p.recent;  // candidates; L > keep >= first + recent
  const int need = p.keep - p.first - p.recent;
  auto key = [&](int t) {
    const Cell c = token_cell<PAGED>(p.page_table, p.max_pages, p.slab, p.num_pages, b, t);
    return float_key(load_dependent(p.weights + ((size_t)c.slab * p.Hkv + h) * p.slab + c.at));
  };
  constexpr uint32_t kZero = 0x80000000u;  // of 0
  uint32_t border = 0xffffffffu;           // nothing is above it
  int left = 0;                            // of the border's keys that are kept
  if (need > 0) {
    uint32_t high = 0u;
    left = need;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
      for (int i = threadIdx.x; i < bins; i += kEvictThreads) hist[i] = 0;
      if (threadIdx.x == 0) s_zero = 0;
      __syncthreads();
      int zeros = 0;
#pragma unroll 4
      for (int t = lo + threadIdx.x; t < hi; t += kEvictThreads) {
        const uint32_t k = key(t);
        if (k == kZero)
          ++zeros;
        else if (pass == 0 || (k ^ high) >> (pass == 1 ? 21 : 10) == 0u)
          atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
      }
      if (pass > 0 && (kZero ^ high) >> (pass == 1 ? 21 : 10) != 0u) zeros = 0;
      zeros = __reduce_add_sync(0xffffffffu, zeros);
      if (lane == 0 && zeros) atomicAdd(&s_zero, zeros);
      __syncthreads();
      if (threadIdx.x == 0) hist[(kZero >> shift) & (bins - 1)] += s_zero;
      __syncthreads();
      // the digit in which the left-th from the top lies: two (one) bins a thread, from the top
      const int per = bins / kEvictThreads;
      int mine = 0;
      for (int i = 0; i < per; ++i) mine += hist[bins - 1 - (threadIdx.x * per + i)];
      int sum = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += up;
      }
      if (lane == 31) s_warp[warp] = sum;
      __syncthreads();
      int before = sum - mine;
      for (int w = 0; w < warp; ++w) before += s_warp[w];
      if (before < left && before + mine >= left) {
        for (int i = 0; i < per; ++i) {
          const int bin = bins - 1 - (threadIdx.x * per + i);
          if (before + hist[bin] >= left) {
            s_digit = bin;
            s_above = before;
            break;
          }
          before += hist[bin];
        }
      }
      __syncthreads();
      high |= (uint32_t)s_digit << shift;
      left -= s_above;
      __syncthreads();
    }
    border = high;
  }
  // every warp's stretch of [0, L), in whole steps of 32
  const int steps = (L + 31) / 32, per = (steps + 31) / 32;
  const int t0 = warp * per * 32, t1 = min(L, t0 + per * 32);
  auto sure = [&](int t, uint32_t k) { return t < lo || t >= hi || k > border; };
  int above = 0, same = 0;
#pragma unroll 4
  for (int t = t0 + lane; t < t1; t += 32) {
    const uint32_t k = t >= lo && t < hi && need > 0 ? key(t) : 0u;
    const bool in = sure(t, k);
    above += in;
    same += !in && need > 0 && k == border;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  same = __reduce_add_sync(0xffffffffu, same);
  if (lane == 0) {
    s_warp[warp] = above;
    s_warp_eq[warp] = same;
  }
  __syncthreads();
  int at = 0, eq = 0;  // kept, and at the border, before this warp's stretch
  for (int w = 0; w < warp; ++w) {
    at += s_warp[w];
    eq += s_warp_eq[w];
  }
  at += min(eq, left);
#pragma unroll 1
  for (int t = t0 + lane; t - lane < t1; t += 32) {
    const bool is = t < t1;
    const uint32_t k = is && t >= lo && t < hi && need > 0 ? key(t) : 0u;
    const bool in = is && sure(t, k), tie = is && !in && need > 0 && k == border;
    const unsigned ties = __ballot_sync(0xffffffffu, tie), below = (1u << lane) - 1u;
    const bool take = in || (tie && eq + __popc(ties & below) < left);
    const unsigned takes = __ballot_sync(0xffffffffu, take);
    if (take) kept[at + __popc(takes & below)] = t;
    at += __popc(takes);
    eq += __popc(ties);
  }
}

constexpr int kMoveThreads = 256;

// A CTA moves the rows' columns [c0, c1) of one (sequence, head, tensor), or the scales and
// weights of one (sequence, head).  In place it goes forward in steps: a row moves to its own
// place or a lower one, so a step's sources lie at or past its targets and past every earlier
// step's; all of a step are loaded before the first is stored.  Byte traffic bounds it: 16 bytes
// a thread, 4 of them in flight.
template <bool PAGED>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int U = 4;
  pdl_wait_primary();
  const int tensors = p.v ? 2 : 1, rolls = tensors * p.columns * p.parts + 1;
  const int unit = blockIdx.x / rolls, role = blockIdx.x % rolls;
  const int b = unit / p.Hkv, h = unit % p.Hkv;
  const int L = seg_len(p.seq_lens, b, p.cap), len = min(L, p.keep);
  const int* kept = p.kept + (size_t)unit * p.keep;
  auto from = [&](int t, bool& good) {
    const Cell c = token_cell<PAGED>(p.page_table, p.max_pages, p.slab, p.num_pages, b, t);
    good = c.good;
    return c;
  };
  auto to = [&](int i, bool& good) {
    if (p.in_place) return from(i, good);
    good = true;
    return Cell{b, i, true};
  };
  const int to_slab = p.in_place ? p.slab : p.out_ctx;

  if (role < rolls - 1) {
    const int part = role % p.parts, column = role / p.parts % p.columns;
    const bool is_v = role / p.parts / p.columns;
    const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.v : p.k);
    uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_out : p.k_out);
    const int chunks = p.row_bytes / 16 / p.columns;  // of a row, here
    const int rows = kMoveThreads / chunks;           // a pass
    const int c = threadIdx.x % chunks, r = threadIdx.x / chunks;
    const long long i_begin = (long long)len * part / p.parts, i_end = (long long)len * (part + 1) / p.parts;
    for (long long i0 = i_begin; i0 < i_end; i0 += rows * U) {
      uint4 w[U];
      int t[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const long long i = i0 + k * rows + r;
        t[k] = r < rows && i < i_end ? load_dependent(kept + i) : -1;
        if (p.in_place && t[k] == i) t[k] = -1;
        w[k] = make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (t[k] >= 0) {
          bool good;
          const Cell s = from(t[k], good);
          if (good)
            w[k] = load_dependent(reinterpret_cast<const uint4*>(
                src + ((s.slab * p.slab + s.at) * p.Hkv + h) * (long long)p.row_bytes) + column * chunks + c);
        }
      if (p.in_place) __syncthreads();
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (t[k] >= 0) {
          bool good;
          const Cell d = to((int)(i0 + k * rows + r), good);
          if (good)
            *(reinterpret_cast<uint4*>(dst + ((d.slab * to_slab + d.at) * p.Hkv + h) * (long long)p.row_bytes) +
              column * chunks + c) = w[k];
        }
    }
    return;
  }
  // numbers: a thread a token
  for (int a = 0; a < 3; ++a) {
    const float* src = a == 0 ? p.ks : a == 1 ? p.vs : p.weights;
    float* dst = a == 0 ? p.ks_out : a == 1 ? p.vs_out : p.weights_out;
    if (!src || !dst) continue;
    for (int i0 = 0; i0 < len; i0 += kMoveThreads * U) {
      float w[U];
      int t[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k * kMoveThreads + threadIdx.x;
        t[k] = i < len ? load_dependent(kept + i) : -1;
        w[k] = 0.f;
        if (t[k] >= 0) {
          bool good;
          const Cell s = from(t[k], good);
          if (good) w[k] = load_dependent(src + ((size_t)s.slab * p.Hkv + h) * p.slab + s.at);
        }
      }
      if (p.in_place) __syncthreads();
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (t[k] >= 0) {
          bool good;
          const Cell d = to(i0 + k * kMoveThreads + threadIdx.x, good);
          if (good) dst[((size_t)d.slab * p.Hkv + h) * to_slab + d.at] = w[k];
        }
    }
    if (a < 2) continue;
    __syncthreads();
    for (int t = len + threadIdx.x; t < (p.in_place ? L : p.out_ctx); t += kMoveThreads) {
      bool good;
      const Cell d = to(t, good);
      if (good) dst[((size_t)d.slab * p.Hkv + h) * to_slab + d.at] = 0.f;
    }
  }
}

}  // namespace da
