// Blocks of a cache: the mean key of each, and the selection of a query's blocks by its
// scores with them.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "device_error.cuh"
#include "ptx.cuh"
#include "seg_kernel.cuh"

namespace da {

// ---------------------------------------------------------------- mean keys

// mean_j = (1 / |j|) sum of the keys of block j's tokens below the length, in fp32, rounded
// once to bf16.  Bytes bound it (a key read once, 1 / block of that written).  A CTA takes
// one block and a share of its row: groups of threads, one 16-byte chunk a thread, take every
// groups-th token each, and are added in order through shared memory.  A step's few blocks
// are cut into shares so that the whole card loads them.  4 prompts of up to 8192 tokens of 8 x 128 (67 MB): 17.6 us,
// 3.8 TB/s in one round of CTAs; the last blocks of 64 sequences: 5.6.
struct MeansParams {
  const __nv_bfloat16* k;
  const int *page_table, *seq_lens;
  __nv_bfloat16* means;  // [B, Hkv, max_blocks, D]
  int B, n, Hkv, D, cap, ctx;
  int page_size, max_pages, num_pages;
  int block, max_blocks;
  int touched;  // blocks a sequence, at most
  int shares;   // CTAs a block; a share is at most kMeansThreads chunks
};
constexpr int kMeansThreads = 256, kMeansTokens = 256;

template <bool PAGED>
__global__ void __launch_bounds__(kMeansThreads) block_means_kernel(const __grid_constant__ MeansParams p) {
  __shared__ float sums[kMeansThreads * 9];     // [group][chunk][8], a chunk 9 apart
  __shared__ unsigned s_row[kMeansTokens];      // where the block's tokens lie, 256 at a time
  pdl_wait_primary();
  pdl_launch_dependents();
  const int share = blockIdx.x % p.shares;
  const long long bj = blockIdx.x / p.shares;
  const int b = (int)(bj / p.touched);
  const int L = seg_len(p.seq_lens, b, p.cap);
  const int j = max(0, L - p.n) / p.block + (int)(bj % p.touched);
  const long long t0 = (long long)j * p.block;
  if (t0 >= L) return;
  const int count = min(p.block, L - (int)t0);
  const int chunks = p.Hkv * p.D / 8, per = (chunks + p.shares - 1) / p.shares;
  const int c0 = share * per, here = min(per, chunks - c0);
  if (here <= 0) return;
  const int groups = kMeansThreads / here, g = threadIdx.x / here, c = threadIdx.x - g * here;
  const uint4* keys = reinterpret_cast<const uint4*>(p.k) + (PAGED ? 0 : ((size_t)b * p.ctx + t0) * chunks) + c0 + c;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int i0 = 0; i0 < count; i0 += kMeansTokens) {
    const int n = min(kMeansTokens, count - i0);
    if constexpr (PAGED) {
      __syncthreads();
      if (threadIdx.x < n) {
        const int t = (int)t0 + i0 + threadIdx.x, col = t / p.page_size;
        int page = load_dependent(p.page_table + (size_t)b * p.max_pages + col);
        if ((unsigned)page >= (unsigned)p.num_pages) {
          atomicOr(&g_error_word, 4u);
          page = 0;
        }
        s_row[threadIdx.x] = (unsigned)(page * (long long)p.page_size + (t - col * p.page_size));
      }
      __syncthreads();
    }
    if (g >= groups) continue;
    constexpr int U = 8;  // loads of a thread in flight
    for (int i = g; i < n; i += U * groups) {
      uint4 w[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int at = i + k * groups;
        w[k] = at < n ? load_dependent(keys + (size_t)(PAGED ? s_row[at] : i0 + at) * chunks) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        s[0] += bf16lo_to_f32(w[k].x);
        s[1] += bf16hi_to_f32(w[k].x);
        s[2] += bf16lo_to_f32(w[k].y);
        s[3] += bf16hi_to_f32(w[k].y);
        s[4] += bf16lo_to_f32(w[k].z);
        s[5] += bf16hi_to_f32(w[k].z);
        s[6] += bf16lo_to_f32(w[k].w);
        s[7] += bf16hi_to_f32(w[k].w);
      }
    }
  }
  if (g < groups)
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[threadIdx.x * 9 + e] = s[e];
  __syncthreads();
  if (g > 0) return;
  for (int o = 1; o < groups; ++o)
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += sums[(o * here + c) * 9 + e];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = s[e] / (float)count;
  const int at = (c0 + c) * 8, h = at / p.D, d = at - h * p.D;
  *reinterpret_cast<uint4*>(p.means + (((size_t)b * p.Hkv + h) * p.max_blocks + j) * p.D + d) =
      make_uint4(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]), pack_bf16x2(s[4], s[5]), pack_bf16x2(s[6], s[7]));
}

// ---------------------------------------------------------------- selection

// For query token i of sequence b (position p = L - n + i) and KV head h, score_j =
// max over the group's heads of <q, mean_j>, j = 0 .. p / block.  The first `first` blocks
// and the last `recent` up to the token's own are taken, and of the others the best scores
// until there are `pick` (ties: the lowest block).  Out: ascending, -1 behind.
//
// The selection is that of the exact scores, as far as the last sentence says.  The products run on the warp-level MMA in
// fp32 (a mean is read once for all 16 rows: heads, and neighbouring tokens where a group
// has few), whose sums are off by mu = D / 16 * 17 * 2^-23 |q| |mean| at most: bf16 products are
// exact, and each of the D / 16 MMAs adds 17 terms, each cut off at 2^-23 of the largest at
// worst.  Where the last block taken and the next differ by more than 2 mu, no block can be on
// the wrong side.  Otherwise those within 2 mu of the border (hardly ever more than two) are
// computed again, each sum with what its additions round off (to 2^-42 of |q| |mean|: the card
// has few 64-bit units), and taken in that order, which compares them pairwise: 512 equal scores take 0.15 ms instead of
// 8 us, 8192 of them 14 ms instead of 26 us.
// Latency bounds it: a mean is 1 / block of its keys, but bins, borders and bits are steps of 0.5 to 1 us that follow one
// another.  16 tokens of 64/8 heads of 128 over up to 512 blocks: 21 us by itself, 11 MB; 500 tokens of 24/4 heads
// of 256 over 128 blocks: 31.
struct SelectParams {
  const __nv_bfloat16 *q, *means;
  const int* seq_lens;
  int* out;  // [B, n, Hkv, pick]
  int B, n, Hq, Hkv, G, cap;
  int block, max_blocks, pick, first, recent;
  int qt;       // query tokens a CTA (cluster)
  int cluster;  // CTAs that share the blocks' scores
};
constexpr int kSelectThreads = 256;   // a CTA; 128 where there are many queries of few blocks
constexpr int kSelectTokens = 16;     // a CTA, at most
constexpr int kSelectBlocks = 8192;

// The squares of 8 bf16 added up.
__device__ __forceinline__ float square_sum(uint4 w, float s) {
  const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(bf16lo_to_f32(e[i]), bf16lo_to_f32(e[i]), s);
    s = fmaf(bf16hi_to_f32(e[i]), bf16hi_to_f32(e[i]), s);
  }
  return s;
}

// s += x, and into e what that rounded off: with t = s + x and v = t - s, exactly (s - (t - v)) + (x - v).
__device__ __forceinline__ void add_exactly(float& s, float& e, float x) {
  const float t = __fadd_rn(s, x), v = __fsub_rn(t, s);
  e += __fadd_rn(__fsub_rn(s, __fsub_rn(t, v)), __fsub_rn(x, v));
  s = t;
}

// float_key of a double: NaN lowest, -0 as 0.
__device__ __forceinline__ unsigned long long double_key(double x) {
  if (x != x) return 0ull;
  const unsigned long long u = (unsigned long long)__double_as_longlong(x == 0.0 ? 0.0 : x);
  return u >> 63 ? ~u : u | 1ull << 63;
}

// mu of a query whose largest square of a head's norm has these bits, among means likewise;
// 2^-110 is for products below fp32's range.
template <int D>
__device__ __forceinline__ float select_slack(uint32_t q2, uint32_t mean2) {
  return D / 16 * 17 * 1.1920929e-7f * sqrtf(__uint_as_float(q2)) * sqrtf(__uint_as_float(mean2)) + 7.7037198e-34f;
}

__device__ __forceinline__ float key_float(uint32_t k) {
  if (k == 0u) return kNegInf;
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// atomicMax at shared-memory address a of the cluster's CTA 0.
__device__ __forceinline__ void max_at_leader(uint32_t a, uint32_t v) {
  asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\tred.shared::cluster.max.u32 [r], %1;\n\t}" ::"r"(a),
               "r"(v)
               : "memory");
}

// The 64-bit scores and numbers of the blocks at the border, the queries' keys and bits.
__host__ __device__ inline size_t select_smem(int qt, int max_blocks) {
  const int words = (max_blocks + 31) / 32;
  return (size_t)max_blocks * 10 + (size_t)qt * (max_blocks + words + 256) * 4 + 16;
}

template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) block_select_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int WARPS = THREADS / 32;
  __shared__ uint32_t s_mean2, s_q2[kSelectTokens];  // bits of the largest squares of norms
  __shared__ uint32_t s_base[kSelectTokens], s_top[kSelectTokens], s_low[kSelectTokens], s_below[kSelectTokens];
  __shared__ int s_shift[kSelectTokens];
  __shared__ int s_left[kSelectTokens], s_open[kSelectTokens], s_count, s_sure, s_busy;
  const int words = (p.max_blocks + 31) / 32;
  unsigned long long* exact = reinterpret_cast<unsigned long long*>(smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(exact + p.max_blocks);
  uint32_t* bits = keys + (size_t)p.qt * p.max_blocks;
  int* hist = reinterpret_cast<int*>(bits + (size_t)p.qt * words);
  uint16_t* list = reinterpret_cast<uint16_t*>(hist + p.qt * 256);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.cluster > 1 ? (int)cluster_rank() : 0;

  const long long unit = blockIdx.x / p.cluster;
  const int tiles = (p.n + p.qt - 1) / p.qt;
  const int i0 = (int)(unit % tiles) * p.qt, h = (int)(unit / tiles % p.Hkv), b = (int)(unit / tiles / p.Hkv);
  const int qn = min(p.qt, p.n - i0);  // query tokens here
  const int rows = qn * p.G;
  const __nv_bfloat16* means = p.means + ((size_t)b * p.Hkv + h) * p.max_blocks * D;
  for (int e = threadIdx.x; e < qn * p.max_blocks; e += THREADS) keys[e] = 0u;
  for (int e = threadIdx.x; e < qn * words; e += THREADS) bits[e] = 0u;
  if (threadIdx.x < kSelectTokens) s_q2[threadIdx.x] = 0u;
  if (threadIdx.x == 0) {
    s_mean2 = 0u;
    s_count = 0;
  }
  if (p.cluster > 1)
    cluster_sync();
  else
    __syncthreads();
  pdl_wait_primary();
  pdl_launch_dependents();

  // scores: 16 query rows against 8 blocks a warp's step.  Element 32 c + 8 t + e of a row is
  // thread t's of the quad, so that rows of both are read 16 bytes at a time; the order of a
  // product's terms is free.  A step's means are loaded a step ahead, the first with the
  // queries and the length (there are max_blocks rows, whatever the length)
  const int step = p.cluster * WARPS, nt0 = rank * WARPS + warp;
  auto load_means = [&](uint4 (&w)[D / 32], int nt, int limit) {
    const int j = nt * 8 + lane / 4;
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      w[c] = j < limit ? load_dependent(reinterpret_cast<const uint4*>(means + (size_t)j * D) + 4 * c + lane % 4)
                       : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 w[D / 32];
  load_means(w, nt0, p.max_blocks);
  const int L = seg_len(p.seq_lens, b, p.cap);
  const int last = L - p.n + i0 + qn - 1;  // position of the last
  const int blocks = last < 0 ? 0 : min(last / p.block + 1, p.max_blocks);
  for (int r0 = 0; r0 < rows; r0 += 16) {
    uint4 a[D / 32][2];
    int qi[2];  // the query token of this thread's two rows, -1: no row
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int row = r0 + lane / 4 + 8 * hf;
      qi[hf] = row < rows ? row / p.G : -1;
      const size_t token = (size_t)b * p.n + i0 + qi[hf];
      const uint4* src = reinterpret_cast<const uint4*>(p.q + (token * p.Hq + h * p.G + row - qi[hf] * p.G) * D) + lane % 4;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) a[c][hf] = qi[hf] >= 0 ? load_dependent(src + 4 * c) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (warp == 0) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float q2 = 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) q2 = square_sum(a[c][hf], q2);
        q2 += __shfl_xor_sync(0xffffffffu, q2, 1);
        q2 += __shfl_xor_sync(0xffffffffu, q2, 2);
        if (lane % 4 == 0 && qi[hf] >= 0) atomicMax(&s_q2[qi[hf]], __float_as_uint(q2));
      }
    }
    if (r0 > 0) load_means(w, nt0, blocks);
    float top2 = 0.f;
    for (int nt = nt0; nt * 8 < blocks; nt += step) {
      float s[4] = {0.f, 0.f, 0.f, 0.f}, m2 = 0.f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        mma_bf16_16816(s, a[c][0].x, a[c][1].x, a[c][0].y, a[c][1].y, w[c].x, w[c].y);
        mma_bf16_16816(s, a[c][0].z, a[c][1].z, a[c][0].w, a[c][1].w, w[c].z, w[c].w);
        m2 = square_sum(w[c], m2);
      }
      load_means(w, nt + step, blocks);
      m2 += __shfl_xor_sync(0xffffffffu, m2, 1);
      m2 += __shfl_xor_sync(0xffffffffu, m2, 2);
      if (nt * 8 + lane / 4 < blocks) top2 = m2 != m2 ? -kNegInf : fmaxf(top2, m2);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = nt * 8 + 2 * (lane % 4) + (e & 1);
        if (qi[e >> 1] >= 0 && col < blocks)
          max_at_leader(smem_u32(keys + (size_t)qi[e >> 1] * p.max_blocks + col), float_key(s[e]));
      }
    }
    if (lane % 4 == 0 && top2 > 0.f) max_at_leader(smem_u32(&s_mean2), __float_as_uint(top2));
  }
  if (p.cluster > 1)
    cluster_sync();
  else
    __syncthreads();
  if (rank != 0) return;

  // what query qi sees and must take
  struct Want {
    int visible, lo, hi, need;  // candidates [lo, hi), of which need are taken; need < 0: every visible block
  };
  auto want = [&](int qi) {
    const int pos = L - p.n + i0 + qi;
    Want w;
    w.visible = pos < 0 ? 0 : min(pos / p.block + 1, p.max_blocks);
    w.lo = min(p.first, w.visible);
    w.hi = max(w.lo, w.visible - p.recent);
    w.need = w.visible <= p.pick ? -1 : p.pick - (w.visible - (w.hi - w.lo));
    return w;
  };
  auto take = [&](int qi, int j) { atomicOr(&bits[qi * words + (j >> 5)], 1u << (j & 31)); };

  // The border of each query: the keys' range is cut into up to 256 equal bins, whose keys are counted;
  // the bin in which the need-th largest lies is the next range, until all keys of that bin are taken
  // (scores spread, so twice as a rule; four times at most).  All queries go side by side, a group of
  // `size` threads each.
  const int size = THREADS / (qn <= 1 ? 1 : qn <= 2 ? 2 : qn <= 4 ? 4 : qn <= 8 ? 8 : 16);
  const int mine = threadIdx.x / size, me = threadIdx.x % size;
  const Want my = mine < qn ? want(mine) : Want{0, 0, 0, 0};
  const uint32_t* key = keys + (size_t)mine * p.max_blocks;
  for (int j = me; j < my.visible; j += size)
    if (my.need < 0 || j < my.lo || j >= my.hi) take(mine, j);
  // the least and the largest number that a group brings, into two words
  auto extremes = [&](uint32_t least, uint32_t most, uint32_t* to_least, uint32_t* to_most) {
    if (size >= 32) {  // a warp is of one group
      least = __reduce_min_sync(0xffffffffu, least);
      most = __reduce_max_sync(0xffffffffu, most);
    }
    if (size < 32 || lane == 0) {
      atomicMin(to_least, least);
      atomicMax(to_most, most);
    }
  };
  if (me == 0 && mine < qn) {
    s_base[mine] = s_low[mine] = 0xffffffffu;
    s_top[mine] = s_below[mine] = 0u;
    s_left[mine] = my.need;
  }
  for (int e = threadIdx.x; e < qn * 256; e += THREADS) hist[e] = 0;
  if (threadIdx.x == 0) s_busy = 0;
  __syncthreads();
  if (my.need > 0) {
    uint32_t least = 0xffffffffu, most = 0u;
    for (int j = my.lo + me; j < my.hi; j += size) {
      least = min(least, key[j]);
      most = max(most, key[j]);
    }
    extremes(least, most, &s_base[mine], &s_top[mine]);
  }
  __syncthreads();
  bool searching = my.need > 0;
  int shift = searching ? max(0, 24 - __clz((int)(s_top[mine] - s_base[mine]))) : 0;
  uint32_t bins = 256u;  // of the range
  for (;;) {
    if (searching) {
      const uint32_t base = s_base[mine];
      if (me == 0) s_shift[mine] = shift;
      for (int j = my.lo + me; j < my.hi; j += size) {
        const uint32_t bin = (key[j] - base) >> shift;
        if (key[j] >= base && bin < bins) atomicAdd(&hist[mine * 256 + bin], 1);
      }
    }
    __syncthreads();
    for (int qi = warp; qi < qn; qi += WARPS) {
      const int left = s_left[qi];
      if (left <= 0) continue;
      // lane l has bins 255 - 8 l .. 248 - 8 l
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = hist[qi * 256 + 255 - 8 * lane - i];
        hist[qi * 256 + 255 - 8 * lane - i] = 0;
        sum += c[i];
      }
      int at = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, at, d);
        if (lane >= d) at += up;
      }
      at -= sum;
      if (at < left && at + sum >= left) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (at < left && at + c[i] >= left) {
            s_base[qi] += (uint32_t)(255 - 8 * lane - i) << s_shift[qi];
            // all keys of this bin are taken: their lowest is the border; one value: some of equal keys are not
            const bool all = at + c[i] == left;
            s_left[qi] = all ? 0 : s_shift[qi] == 0 ? -(left - at) : left - at;
            if (!all && s_shift[qi] > 0) s_busy = 1;
            break;
          }
          at += c[i];
        }
      }
      __syncwarp();
    }
    __syncthreads();
    const bool busy = s_busy;
    searching = searching && s_left[min(mine, qn - 1)] > 0;
    bins = shift >= 8 ? 256u : 1u << shift;
    shift = max(0, shift - 8);
    __syncthreads();
    if (threadIdx.x == 0) s_busy = 0;
    if (!busy) break;
  }
  // the lowest key taken, and the largest below it; a query with something left has equal keys on both sides
  if (my.need > 0) {
    const uint32_t from = s_base[mine];
    uint32_t low = 0xffffffffu, below = 0u;
    for (int j = my.lo + me; j < my.hi; j += size) {
      const uint32_t k = key[j];
      if (k >= from)
        low = min(low, k);
      else
        below = max(below, k);
    }
    extremes(low, below, &s_low[mine], &s_below[mine]);
  }
  __syncthreads();
  if (my.need > 0) {
    const float mu = select_slack<D>(s_q2[mine], s_mean2);
    const uint32_t low = s_low[mine];
    if (s_left[mine] == 0 && key_float(low) - key_float(s_below[mine]) > 2.f * mu) {
      for (int j = my.lo + me; j < my.hi; j += size)
        if (key[j] >= low) take(mine, j);
    } else if (me == 0) {
      s_open[atomicAdd(&s_count, 1)] = mine;
    }
  }
  __syncthreads();

  // queries whose border is too close to call
  const int open = s_count;
  for (int o = 0; o < open; ++o) {
    const int qi = s_open[o];
    const Want w = want(qi);
    const uint32_t* key = keys + (size_t)qi * p.max_blocks;
    const float border = key_float(s_low[qi]), mu = select_slack<D>(s_q2[qi], s_mean2);
    __syncthreads();
    if (threadIdx.x == 0) s_count = s_sure = 0;
    __syncthreads();
    for (int j = w.lo + threadIdx.x; j < w.hi; j += THREADS) {
      const float s = key_float(key[j]);
      if (s > border + 2.f * mu) {
        take(qi, j);
        atomicAdd(&s_sure, 1);
      } else if (!(s < border - 2.f * mu)) {
        const int c = atomicAdd(&s_count, 1);
        list[c] = (uint16_t)j;
        exact[c] = 0ull;
      }
    }
    __syncthreads();
    // half a warp a (candidate, head): the largest of the heads' scores, ordered by their bits
    const int count = s_count, left = w.need - s_sure;
    const __nv_bfloat16* q = p.q + (((size_t)b * p.n + i0 + qi) * p.Hq + h * p.G) * D;
    const int half = lane >> 4, hl = lane & 15;
    for (int e0 = 2 * warp; e0 < count * p.G; e0 += 2 * WARPS) {
      const int e = min(e0 + half, count * p.G - 1), c = e / p.G, g = e - c * p.G;
      const uint4* a = reinterpret_cast<const uint4*>(q + g * D) + hl;
      const uint4* m = reinterpret_cast<const uint4*>(means + (size_t)list[c] * D) + hl;
      float s = 0.f, e2 = 0.f;  // a sum and what its additions rounded off
#pragma unroll
      for (int d = 0; d < (D + 127) / 128; ++d) {
        if (D >= 128 || hl < D / 8) {
          const uint4 x = load_dependent(a + 16 * d), y = load_dependent(m + 16 * d);
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            add_exactly(s, e2, bf16lo_to_f32(xs[i]) * bf16lo_to_f32(ys[i]));
            add_exactly(s, e2, bf16hi_to_f32(xs[i]) * bf16hi_to_f32(ys[i]));
          }
        }
      }
#pragma unroll
      for (int d = 8; d; d >>= 1) {
        const float os = __shfl_xor_sync(0xffffffffu, s, d), oe = __shfl_xor_sync(0xffffffffu, e2, d);
        add_exactly(s, e2, os);
        e2 += oe;
      }
      if (hl == 0) atomicMax(&exact[c], double_key((double)s + (double)(s - s == 0.f ? e2 : 0.f)));
    }
    __syncthreads();
    for (int c = threadIdx.x; c < count; c += THREADS) {
      const unsigned long long s = exact[c];
      const int j = list[c];
      int before = 0;
      for (int i = 0; i < count; ++i) before += exact[i] > s || (exact[i] == s && list[i] < j);
      if (before < left) take(qi, j);
    }
    __syncthreads();
  }

  // the numbers of the bits, ascending
  for (int qi = warp; qi < qn; qi += THREADS / 32) {
    int* dst = p.out + (((size_t)b * p.n + i0 + qi) * p.Hkv + h) * p.pick;
    int at = 0;
    for (int w0 = 0; w0 < words; w0 += 32) {
      uint32_t w = w0 + lane < words ? bits[qi * words + w0 + lane] : 0u;
      const int mine = __popc(w);
      int sum = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += up;
      }
      int k = at + sum - mine;
      while (w) {
        if (k < p.pick) dst[k] = (w0 + lane) * 32 + __ffs(w) - 1;
        ++k;
        w &= w - 1;
      }
      at += __shfl_sync(0xffffffffu, sum, 31);
    }
    for (int k = at + lane; k < p.pick; k += 32) dst[k] = -1;
  }
}

}  // namespace da
