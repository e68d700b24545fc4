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
  int cluster;  // CTAs that share a (sequence, head)'s weights
  int keys;     // of them that a CTA's shared memory holds
  int parts;    // CTAs that share a (sequence, head, tensor)'s rows (in place: 1)
  int columns;  // CTAs that share its rows' bytes
};

constexpr int kEvictThreads = 512;

// Adds at shared-memory address a of the cluster's CTA `rank`, or stores there.
__device__ __forceinline__ void add_at(uint32_t a, int rank, int v) {
  asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, %1;\n\tred.shared::cluster.add.u32 [r], %2;\n\t}" ::"r"(a),
               "r"(rank), "r"(v)
               : "memory");
}
__device__ __forceinline__ void store_at(uint32_t a, int rank, int v) {
  asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, %1;\n\tst.shared::cluster.u32 [r], %2;\n\t}" ::"r"(a),
               "r"(rank), "r"(v)
               : "memory");
}

// The candidates are the positions [first, L - recent); a cluster's CTAs take a stretch of them
// each, and keep its keys in shared memory (as long as they fit: `keys`).  The need-th largest key
// is found 11, 11 and 10 bits at a time: each CTA counts its keys of each digit, CTA 0 adds the
// counts up and finds the digit in which the need-th lies.  Zeros, of which there may be very
// many, are counted in registers.  Then each warp counts what it keeps of its stretch, and after
// one sum over the warps and one over the CTAs writes it in place.
// Latency bounds it: one pass over the weights, 6 to 8 meetings of the cluster.  32768 weights of 8 heads: 13 us,
// 16 x 8 x <= 8192 in pages: 21 to 25.  Clusters for up to 4 CTAs an SM instead of 2 and, below, 4 rows a thread
// instead of 8 took a call with its read back from 65 to 60 us.
template <bool PAGED>
__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t s_keys[];
  constexpr int WARPS = kEvictThreads / 32;
  __shared__ int hist[2048], total[2048];  // this CTA's counts; the cluster's (CTA 0)
  __shared__ int s_warp[WARPS], s_warp_same[WARPS], s_digit[3], s_above[3], s_done[3];
  __shared__ int s_kept[8], s_same[8];  // of every CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.cluster > 1 ? (int)cluster_rank() : 0;
  auto meet = [&]() {
    if (p.cluster > 1)
      cluster_sync();
    else
      __syncthreads();
  };
  for (int i = threadIdx.x; i < 2048; i += kEvictThreads) hist[i] = total[i] = 0;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int unit = blockIdx.x / p.cluster, b = unit / p.Hkv, h = unit % p.Hkv;
  const int L = seg_len(p.seq_lens, b, p.cap);
  int* kept = p.kept + (size_t)unit * p.keep;
  if (rank == 0 && h == 0 && threadIdx.x == 0) p.new_lens[b] = min(L, p.keep);
  if (L <= p.keep) {  // (all of the cluster)
    for (int i = rank * kEvictThreads + threadIdx.x; i < p.keep; i += p.cluster * kEvictThreads) kept[i] = i < L ? i : -1;
    return;
  }
  const int hi = L - p.recent;                        // L > keep >= first + recent
  const int need = p.keep - p.first - p.recent;       // of the candidates, which are more
  const int share = (hi - p.first + p.cluster - 1) / p.cluster;
  const int lo = min(hi, p.first + rank * share), count = min(hi, lo + share) - lo;
  // forced ones
  for (int i = rank * kEvictThreads + threadIdx.x; i < p.first + p.recent; i += p.cluster * kEvictThreads)
    kept[i < p.first ? i : i + need] = i < p.first ? i : hi + i - p.first;
  auto read = [&](int i) {
    const Cell c = token_cell<PAGED>(p.page_table, p.max_pages, p.slab, p.num_pages, b, lo + i);
    return float_key(load_dependent(p.weights + ((size_t)c.slab * p.Hkv + h) * p.slab + c.at));
  };
  const int held = min(count, p.keys);
#pragma unroll 8
  for (int i = threadIdx.x; i < held; i += kEvictThreads) s_keys[i] = read(i);
  auto key = [&](int i) { return i < held ? s_keys[i] : read(i); };
  meet();

  constexpr uint32_t kZero = 0x80000000u;  // the key of 0
  uint32_t border = 0xffffffffu;           // keys above it are kept, and the first `left` of those that are it
  int left = 0;
  if (need > 0) {
    uint32_t high = 0u;
    left = need;
    bool done = false;
#pragma unroll 1
    for (int pass = 0; pass < 3 && !done; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
      const int known = pass == 1 ? 21 : 10;  // bits below the digits found so far
      auto mine = [&](uint32_t k) { return pass == 0 || (k ^ high) >> known == 0u; };
      int zeros = 0;
#pragma unroll 4
      for (int i = threadIdx.x; i < count; i += kEvictThreads) {
        const uint32_t k = key(i);
        if (k == kZero)
          ++zeros;
        else if (mine(k))
          atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
      }
      if (!mine(kZero)) zeros = 0;
      zeros = __reduce_add_sync(0xffffffffu, zeros);
      if (lane == 0 && zeros) atomicAdd(&hist[(kZero >> shift) & (bins - 1)], zeros);
      __syncthreads();
      int* sums = hist;
      if (p.cluster > 1) {
        for (int i = threadIdx.x; i < bins; i += kEvictThreads) {
          if (hist[i]) add_at(smem_u32(&total[i]), 0, hist[i]);
          hist[i] = 0;
        }
        cluster_sync();
        sums = total;
      }
      if (rank == 0) {
        // the digit in which the left-th from the top lies: 4 (2) bins a thread, from the top
        const int per = bins / kEvictThreads;
        int c[4], mine4 = 0;
        for (int i = 0; i < per; ++i) {
          c[i] = sums[bins - 1 - (threadIdx.x * per + i)];
          sums[bins - 1 - (threadIdx.x * per + i)] = 0;
          mine4 += c[i];
        }
        int sum = mine4;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, sum, d);
          if (lane >= d) sum += up;
        }
        if (lane == 31) s_warp[warp] = sum;
        __syncthreads();
        int before = __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0) + sum - mine4;
        if (before < left && before + mine4 >= left) {
          int i = 0;
          while (before + c[i] < left) before += c[i++];
          const int digit = bins - 1 - (threadIdx.x * per + i), all = before + c[i] == left;  // all of the digit's are kept
          for (int r = 0; r < p.cluster; ++r) {
            store_at(smem_u32(&s_digit[pass]), r, digit);
            store_at(smem_u32(&s_above[pass]), r, before);
            store_at(smem_u32(&s_done[pass]), r, all);
          }
        }
      }
      meet();
      high |= (uint32_t)s_digit[pass] << shift;
      left -= s_above[pass];
      done = s_done[pass];
    }
    // where all keys of the last digit are kept, the border lies below the lowest they can be (which is
    // not 0: as many candidates as are needed are not all of them)
    border = done ? high - 1u : high;
    if (done) left = 0;
  }
  // every warp's stretch, in whole steps of 32
  const int steps = (count + 31) / 32, per = (steps + WARPS - 1) / WARPS;
  const int i0 = warp * per * 32, i1 = min(count, i0 + per * 32);
  int above = 0, same = 0;
  if (need > 0) {
#pragma unroll 4
    for (int i = i0 + lane; i < i1; i += 32) {
      const uint32_t k = key(i);
      above += k > border;
      same += k == border;
    }
  }
  above = __reduce_add_sync(0xffffffffu, above);
  same = __reduce_add_sync(0xffffffffu, same);
  if (lane == 0) {
    s_warp[warp] = above;
    s_warp_same[warp] = same;
  }
  __syncthreads();
  const int w_above = lane < WARPS ? s_warp[lane] : 0, w_same = lane < WARPS ? s_warp_same[lane] : 0;
  int at = __reduce_add_sync(0xffffffffu, lane < warp ? w_above : 0), eq = __reduce_add_sync(0xffffffffu, lane < warp ? w_same : 0);
  if (p.cluster > 1) {
    const int all_above = __reduce_add_sync(0xffffffffu, w_above), all_same = __reduce_add_sync(0xffffffffu, w_same);
    if (warp == 0 && lane < p.cluster) {
      store_at(smem_u32(&s_kept[rank]), lane, all_above);
      store_at(smem_u32(&s_same[rank]), lane, all_same);
    }
    cluster_sync();
    at += __reduce_add_sync(0xffffffffu, lane < rank ? s_kept[lane & 7] : 0);
    eq += __reduce_add_sync(0xffffffffu, lane < rank ? s_same[lane & 7] : 0);
  }
  if (need == 0) return;
  at += p.first + min(eq, left);
#pragma unroll 1
  for (int i = i0 + lane; i - lane < i1; i += 32) {
    const uint32_t k = i < i1 ? key(i) : 0u;
    const bool in = i < i1 && k > border, tie = i < i1 && k == border;
    const unsigned ties = __ballot_sync(0xffffffffu, tie), below = (1u << lane) - 1u;
    const bool take = in || (tie && eq + __popc(ties & below) < left);
    const unsigned takes = __ballot_sync(0xffffffffu, take);
    if (take) kept[at + __popc(takes & below)] = lo + i;
    at += __popc(takes);
    eq += __popc(ties);
  }
}

constexpr int kMoveThreads = 256;

// A CTA moves the rows' columns [c0, c1) of one (sequence, head, tensor), or the scales or the
// weights of one (sequence, head).  In place it goes forward in steps: a row moves to its own
// place or a lower one, so a step's sources lie at or past its targets and past every earlier
// step's; all of a step are loaded before the first is stored.  Byte traffic bounds it, and for
// few rows the chain of kept position, page and row: 16 bytes a thread, 4 of them in flight.  2 x 16 x 8 x 1024
// rows of 128 bytes, in place, in pages: 21 us by itself (34 MB gathered, 34 stored).
template <bool PAGED>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int U = 4;
  pdl_wait_primary();
  const int tensors = p.v ? 2 : 1, copies = tensors * p.columns * p.parts, rolls = copies + 3;
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

  if (role < copies) {
    const int part = role % p.parts, column = role / p.parts % p.columns;
    const bool is_v = role / p.parts / p.columns;
    const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.v : p.k);
    uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_out : p.k_out);
    const int chunks = p.row_bytes / 16 / p.columns;  // of a row, here
    const int rows = kMoveThreads / chunks;           // a pass
    const int c = threadIdx.x % chunks, r = threadIdx.x / chunks;
    // a row's place: its page's (sequence's) and, in it, its own
    const long long head = (long long)h * p.row_bytes + (column * chunks + c) * 16, row_step = (long long)p.Hkv * p.row_bytes;
    const long long src_slab = row_step * p.slab, dst_slab = row_step * to_slab;
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
            w[k] = load_dependent(reinterpret_cast<const uint4*>(src + s.slab * src_slab + s.at * row_step + head));
        }
      if (p.in_place) __syncthreads();
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (t[k] >= 0) {
          bool good;
          const Cell d = to((int)(i0 + k * rows + r), good);
          if (good)
            *reinterpret_cast<uint4*>(dst + d.slab * dst_slab + d.at * row_step + head) = w[k];
        }
    }
    return;
  }
  // numbers: a thread a token
  {
    const int a = role - copies;
    const float* src = a == 0 ? p.weights : a == 1 ? p.ks : p.vs;
    float* dst = a == 0 ? p.weights_out : a == 1 ? p.ks_out : p.vs_out;
    if (!dst || (!src && len > 0)) return;
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
    if (a > 0) return;
    __syncthreads();
    for (int t = len + threadIdx.x; t < (p.in_place ? L : p.out_ctx); t += kMoveThreads) {
      bool good;
      const Cell d = to(t, good);
      if (good) dst[((size_t)d.slab * p.Hkv + h) * to_slab + d.at] = 0.f;
    }
  }
}

}  // namespace da
