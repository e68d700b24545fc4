// Attention of query rows over lists of cached tokens, for few rows a KV head: the tokens
// [base, L) of a sequence, the first base tokens that a batch shares, or the blocks that
// were selected for a query.  (A unit of a sequence's rows goes along all of its tokens, those that none of its rows sees
// among them: for new prompts it is slow.)  The tokens' bytes should bound it, so a CTA reads each key and
// value once for its 8 or 16 rows.
//
// The warp-level MMA of this card gives 256 products a cycle and SM (a 16 x 8 x 16 step every
// 32 cycles a scheduler, measured), a sixteenth of tcgen05's, and would bound it first if its 16
// rows were the queries, of which a group has 4 to 8.  So the tokens are its 16 rows and the
// queries its 8 columns:
//     S^T = K Q^T (16 tokens x 8 rows),   O^T += V^T P^T (D x 8 rows),
// D / 8 steps for 16 tokens and 8 rows, 1 KB of keys and values a 1024 / D steps; P^T is S^T's
// accumulator, transposed 8 x 8 at a time.
//
// The 4 warps of a CTA take 16 tokens each of every tile of 64 and run on their own, with
// no barrier between them: a warp looks up where its 16 tokens lie two tiles ahead (they start at a
// multiple of 16 and pages hold whole 16s, so their rows are equally far apart: one look-up and an
// addition a row; a look-up a row made half of the instructions), copies their rows into its own ring
// (cp.async; rows that do not exist are zeros there), keys and values in turn, and keeps a running
// maximum m, sum l and output O of its tokens,
//     O = sum_t 2^(s_t - m) v_t,   l = sum_t 2^(s_t - m),   s_t = scale log2(e) <q, k_t>.
// Where a unit ends the warps' four (m, l, O) are joined through shared memory.  m is only raised
// when a score passes it by more than 8; it cancels in O / l.
//
// Ranges are ragged: their tiles are cut evenly over the CTAs (seg_plan.cuh), each piece is
// written as a partial, and a merge kernel joins them, with the prefix's.  Blocks units all
// have as many tiles: a cluster of 1 to 16 CTAs takes a unit, each CTA its share of the tiles, and
// joins it through distributed shared memory.
//
// Measured: 64 of 64 tokens of 16 sequences, 64/8 heads of 128, pages of 32: 258 MB in 52 us by itself (63% of HBM's rate:
// its loads' latency); 16 of 64 for each of 500 tokens, 24/4 heads of 256: 2.1 GB through L2 in 200 us, next to 113 of MMAs;
// the rests of 64 sequences behind a prefix (71 MB): 15 us after a start of 4.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "device_error.cuh"
#include "ptx.cuh"
#include "seg_plan.cuh"

namespace da {

constexpr float kNegInf = -__builtin_huge_valf();

// Ordered as the numbers: NaN lowest, -0 as 0.
__device__ __forceinline__ uint32_t float_key(float f) {
  if (f != f) return 0u;
  const uint32_t u = __float_as_uint(f == 0.f ? 0.f : f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSegCluster = 16;  // CTAs that may share a blocks unit
constexpr int kSegLens = 512;  // lengths that a CTA copies to its shared memory

// Ranges of one new token each (every row of a unit sees all of its tokens), of several or of a whole batch's
// prefix (a row may see fewer), and blocks.
enum SegKind { kSegRange = 0, kSegBlocks = 1, kSegEdges = 2 };

struct SegParams {
  const __nv_bfloat16* q;      // [B, n, Hq, D]
  const __nv_bfloat16 *k, *v;  // contiguous [B, ctx, Hkv, D] (token t in row t - base), or pools
  const __nv_bfloat16 *kp, *vp;  // the shared prefix's cache, contiguous: [base, Hkv, D]
  const int* seq_lens;         // prefix included; null: cap
  const int *page_table, *prefix_table;
  const int* blocks;           // [B, n, Hkv, pick]
  __nv_bfloat16* out;          // like q
  float* part_o;               // [slots][ru][D] (seg_plan.cuh; ranges only)
  float2* part_ml;             // [slots][ru]: m, l
  const float* tc_o;           // [slabs][Hkv][B n G][D]: the prefix's partials, where another kernel made them
  const float2* tc_ml;
  int slabs;
  int B, n, Hq, Hkv, G;
  int base;                    // tokens of the shared prefix; the rests' tiles start at the multiple of 16 below
  int cap;                     // longest sequence
  int ctx;
  int page_size, max_pages, num_pages;
  int block, pick;
  int ru;                      // query rows of a unit: 8 or 16
  int rt, rt_prefix;           // units a sequence's KV head (rows over ru), and of the prefix's (0: none here)
  int ctas;                    // of seg_kernel; ranges: the plan's n
  int cluster;                 // CTAs that share a blocks unit
  int beside;                  // the kernel before is the prefix's: seg_kernel runs beside it and waits for it at its end
  float scale_log2;
};

// A row where a unit's warps are joined: their factors, and its place in the output (-1: no row).
struct FoldRow {
  float f[4];
  long long out;
};

template <int D, int NT, int KIND = kSegRange>
struct SegGeo {
  static constexpr int WARPS = 4, THREADS = 32 * WARPS;
  static constexpr int ROWS = 8 * NT;           // query rows of a unit
  static constexpr int ROWB = 2 * D;            // a row of K or V
  static constexpr int GRAN = 16 * ROWB;        // 16 tokens of one of them; also 8 rows of O in fp32
  static constexpr int NG = D == 64 ? 5 : D == 256 ? 2 : 3;  // of them in a warp's ring
  static constexpr int WARP_BYTES = NG * GRAN;
  static constexpr int OFF_ML = WARPS * WARP_BYTES;
  static constexpr int OFF_FOLD = OFF_ML + WARPS * ROWS * 8;
  static constexpr int OFF_LENS = OFF_FOLD + ROWS * (int)sizeof(FoldRow);
  static constexpr int OFF_RES = OFF_LENS + kSegLens * 4;  // blocks: this CTA's (m, l) and O, for the cluster
  static constexpr int OFF_ODD = OFF_RES;                  // edges: see there
  static constexpr int SMEM =
      OFF_RES + (KIND == kSegBlocks ? ROWS * (8 + D * 4) : KIND == kSegEdges ? 4 + ROWS * (D + 4) : 0);
  static constexpr int PER_SM = D == 256 ? 3 : NT == 1 ? 4 : 3;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// A word or four at shared-memory address a of the cluster's CTA `rank`.
template <typename T>
__device__ __forceinline__ T load_at(uint32_t a, int rank);
template <>
__device__ __forceinline__ float2 load_at<float2>(uint32_t a, int rank) {
  float2 v;
  asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %2, %3;\n\tld.shared::cluster.v2.f32 {%0, %1}, [r];\n\t}"
               : "=f"(v.x), "=f"(v.y)
               : "r"(a), "r"(rank)
               : "memory");
  return v;
}
template <>
__device__ __forceinline__ float4 load_at<float4>(uint32_t a, int rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %4, %5;\n\tld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [r];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(a), "r"(rank)
      : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Copies 16 bytes, or writes as many zeros and reads nothing.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ int seg_len(const int* lens, int b, int cap) {
  const int L = lens ? load_dependent(lens + b) : cap;
  return L < 0 ? 0 : L < cap ? L : cap;
}

// The lengths where a CTA reads them often: in its shared memory, if they fit.  The CTA executes it.
template <int THREADS>
__device__ __forceinline__ const int* seg_stage_lens(const SegParams& p, int* to) {
  if (!p.seq_lens || p.B > kSegLens) return p.seq_lens;
  for (int b = threadIdx.x; b < p.B; b += THREADS) to[b] = load_dependent(p.seq_lens + b);
  __syncthreads();
  return to;
}

// A unit: ru query rows (from row ru r of its rows) of KV head h, and its tokens.
struct SegUnit {
  int b, i, h, r;
  int prefix;  // rows of the whole batch, over the shared prefix
  int len;     // the sequence's length (of a prefix unit: unused)
  int end;     // tokens [base or 0, end)
  int tiles;
  int id;
};

template <int KIND>
struct SegWalk {
  const SegParams& p;
  const int* lens;  // seq_lens, or the CTA's copy
  long long all;  // tiles of the line
  int tp;         // tiles of a prefix unit, or of a blocks unit
  int used;       // CTAs that have some
  int lo, hi;     // blocks: this CTA's tiles of a unit
  int units;      // blocks

  __device__ __forceinline__ SegWalk(const SegParams& p_, const int* lens_)
      : p(p_), lens(lens_), all(0), tp(0), used(0), lo(0), hi(0), units(0) {
    if constexpr (KIND == kSegBlocks) {
      tp = (p.pick * p.block + kTile - 1) / kTile;
      const int rank = blockIdx.x % p.cluster;
      lo = tp * rank / p.cluster;
      hi = tp * (rank + 1) / p.cluster;
      units = p.B * p.n * p.Hkv * p.rt;
    } else {
      tp = p.rt_prefix ? (p.base + kTile - 1) / kTile : 0;
      all = seg_sums(lens, p.B, p.cap, p.base & ~15, 0).all * p.Hkv * p.rt + prefix_tiles();
      used = seg_used(all, p.ctas);
    }
  }
  // The tiles [x0, x1) of a CTA, of ranges in the line; false if there are none.
  __device__ __forceinline__ bool range(int c, long long& x0, long long& x1) const {
    if constexpr (KIND == kSegBlocks) {
      const int first = c / p.cluster, step = p.ctas / p.cluster;
      x0 = 0;
      x1 = first < units ? (long long)((units - first + step - 1) / step) * (hi - lo) : 0;
      return x1 > 0;
    } else {
      if (c >= used) return false;
      x0 = seg_start(all, used, c);
      x1 = seg_start(all, used, c + 1);
      return true;
    }
  }
  __device__ __forceinline__ long long prefix_tiles() const { return (long long)p.Hkv * p.rt_prefix * tp; }
  // Of this CTA: the first tile of a unit that it starts, and the end of its tiles.
  __device__ __forceinline__ int first_tile() const { return KIND == kSegBlocks ? lo : 0; }
  __device__ __forceinline__ int end_tile(const SegUnit& u) const { return KIND == kSegBlocks ? hi : u.tiles; }

  // A blocks unit by number.
  __device__ __forceinline__ SegUnit blocks_unit(int id) const {
    SegUnit u;
    u.id = id;
    u.r = id % p.rt;
    id /= p.rt;
    u.h = id % p.Hkv;
    id /= p.Hkv;
    u.i = id % p.n;
    u.b = id / p.n;
    u.prefix = 0;
    u.tiles = tp;
    u.len = seg_len(lens, u.b, p.cap);
    u.end = max(0, u.len - p.n + 1 + u.i);
    return u;
  }
  __device__ __forceinline__ SegUnit prefix_unit(int id) const {
    SegUnit u = {};
    u.id = id;
    u.h = id / p.rt_prefix;
    u.r = id % p.rt_prefix;
    u.prefix = 1;
    u.tiles = tp;
    u.end = p.base;
    return u;
  }
  __device__ __forceinline__ SegUnit range_unit(int b, int h, int r) const {
    SegUnit u;
    u.b = b;
    u.i = 0;
    u.h = h;
    u.r = r;
    u.prefix = 0;
    u.len = u.end = seg_len(lens, b, p.cap);
    u.tiles = seg_tiles(u.end, p.cap, p.base & ~15);
    u.id = p.Hkv * p.rt_prefix + (b * p.Hkv + h) * p.rt + r;
    return u;
  }
  // The unit of tile x (x < all; blocks: the CTA's first), j: the tile's place in it.  The warp executes it.
  __device__ __forceinline__ SegUnit at(long long x, int& j) const {
    if constexpr (KIND == kSegBlocks) {
      j = lo;
      return blocks_unit((int)blockIdx.x / p.cluster);
    } else {
      const long long wp = prefix_tiles();
      if (x < wp) {
        const int id = (int)seg_div(x, tp);
        j = (int)(x - (long long)id * tp);
        return prefix_unit(id);
      }
      x -= wp;
      const int hr = p.Hkv * p.rt;
      const SegAt f = seg_find(lens, p.B, p.cap, p.base & ~15, seg_div(x, hr));
      const int tb = seg_tiles(seg_len(lens, f.b, p.cap), p.cap, p.base & ~15);
      const long long in = x - f.start * hr;
      const int w = (int)seg_div(in, tb);
      j = (int)(in - (long long)w * tb);
      return range_unit(f.b, w / p.rt, w % p.rt);
    }
  }
  // The next unit that has tiles; there is one.
  __device__ __forceinline__ SegUnit next(const SegUnit& u) const {
    if constexpr (KIND == kSegBlocks) {
      return blocks_unit(u.id + p.ctas / p.cluster);
    } else {
      int b = u.b, h = u.h, r = u.r + 1;
      if (u.prefix) {
        if (u.id + 1 < p.Hkv * p.rt_prefix) return prefix_unit(u.id + 1);
        b = 0;
        h = 0;
        r = 0;
      } else {
        if (r == p.rt) {
          r = 0;
          ++h;
        }
        if (h == p.Hkv) {
          h = 0;
          ++b;
        }
      }
      SegUnit v = range_unit(b, h, r);
      while (v.tiles == 0 && b + 1 < p.B) v = range_unit(++b, 0, 0);
      return v;
    }
  }
};

// 16 tokens: the element offset of the first one's row of head h in the cache (or the prefix's), the rest
// Hkv D apart, and which of them there are (bit i: token i).  A page outside the pool is flagged and
// page 0 read instead.  The same in every lane.
struct SegGroup {
  long long off;
  uint32_t live;
};
template <int D, bool PAGED, int KIND>
__device__ __forceinline__ SegGroup seg_group(const SegParams& p, const SegUnit& u, int at) {
  int t;  // the first token
  if constexpr (KIND == kSegBlocks) {
    const int e = at / p.block;
    if (e >= p.pick) return {0, 0u};
    const int id = load_dependent(p.blocks + (((size_t)u.b * p.n + u.i) * p.Hkv + u.h) * p.pick + e);
    if (id < 0 || id > (u.end - 1) / p.block) return {0, 0u};
    t = id * p.block + (at - e * p.block);
  } else {
    t = at + (u.prefix ? 0 : p.base & ~15);
  }
  const int n = u.end - t;
  if (n <= 0) return {0, 0u};
  uint32_t live = n < 16 ? (1u << n) - 1u : 0xffffu;
  if (KIND != kSegBlocks && !u.prefix && t < p.base) live &= 0xffffu << (p.base - t);
  if constexpr (PAGED) {
    const int col = t / p.page_size;
    int page = live ? load_dependent(u.prefix ? p.prefix_table + col : p.page_table + (size_t)u.b * p.max_pages + col) : 0;
    if ((unsigned)page >= (unsigned)p.num_pages) {
      atomicOr(&g_error_word, 4u);
      page = 0;
    }
    return {(((long long)page * p.page_size + (t - col * p.page_size)) * p.Hkv + u.h) * D, live};
  } else {
    const long long row = u.prefix ? t : (long long)u.b * p.ctx + (t - p.base);
    return {(row * p.Hkv + u.h) * D, live};
  }
}

// Row rr of a unit: its query token (over the batch), head in the group, and how many tokens
// it sees; false past the unit's rows.
template <int KIND>
__device__ __forceinline__ bool seg_query(const SegParams& p, const int* lens, const SegUnit& u, int rr, int& token, int& g,
                                          int& lim) {
  const int row = u.r * p.ru + rr;
  if constexpr (KIND == kSegBlocks) {
    token = u.b * p.n + u.i;
    g = row;
    lim = u.end;
    return row < p.G;
  } else {
    const int i = row / p.G;  // of the batch's tokens, or the sequence's
    g = row - i * p.G;
    token = u.prefix ? i : u.b * p.n + i;
    if (i >= (u.prefix ? p.B * p.n : p.n)) {
      lim = 0;
      return false;
    }
    const int b = u.prefix ? i / p.n : u.b;
    lim = (u.prefix ? seg_len(lens, b, p.cap) : u.len) - p.n + 1 + (u.prefix ? i - b * p.n : i);
    return true;
  }
}

// The sum of values that are not finite: infinities of one sign, else NaN; 0 of none.
__device__ __forceinline__ float odd_value(uint32_t marks) {
  marks &= 7u;
  return marks == 0u ? 0.f : marks == 1u ? -kNegInf : marks == 2u ? kNegInf : __int_as_float(0x7fffffff);
}

// An 8 x 8 matrix of 16-bit elements, lane l holding row l / 4, columns 2 (l % 4) and the next: its transpose.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, bool PAGED, int KIND, int NT>
__global__ void __launch_bounds__(SegGeo<D, NT, KIND>::THREADS, SegGeo<D, NT, KIND>::PER_SM)
    seg_kernel(const __grid_constant__ SegParams p) {
  using Gm = SegGeo<D, NT, KIND>;
  constexpr int NG = Gm::NG;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring_s = smem_u32(smem + warp * Gm::WARP_BYTES);

  // Beside the prefix's kernel there is nothing to wait for: it has written nothing that is read
  // here, and lets this kernel start after its own wait for what came before.  The kernels after this
  // one wait for this one alone, so it may not end before that one does.
  if (!p.beside) pdl_wait_primary();
  pdl_launch_dependents();
  const SegWalk<KIND> walk(p, seg_stage_lens<Gm::THREADS>(p, reinterpret_cast<int*>(smem + Gm::OFF_LENS)));
  long long x0, x1;
  if (!walk.range(blockIdx.x, x0, x1)) {
    if (p.beside) pdl_wait_primary();
    return;
  }

  // the load side: where this warp's tokens of the next tile to copy lie, and of the one after it; lu
  // and lj are the unit and tile of the latter
  int lj;
  SegUnit lu = walk.at(x0, lj);
  const SegUnit u0 = lu;
  const int start = lj;
  long long lx = x0;
  auto look_up = [&]() { return seg_group<D, PAGED, KIND>(p, lu, lj * kTile + warp * 16); };
  SegGroup now = look_up(), then = {0, 0u};
  unsigned long long lives = 0ull;  // of the last four tiles, tile x in bits 16 (x % 4) on
  int ls = 0;          // the next granule's slot
  bool lv = false;     // it is of values
  bool ahead = false;  // `then` is of the tile after lx
  const int row_step = p.Hkv * D;
  auto issue = [&]() {
    if (lx < x1) {
      if (!ahead) {  // (once a tile, with its keys)
        ahead = true;
        then.live = 0u;
        if (lx + 1 < x1) {
          if (++lj == walk.end_tile(lu)) {
            lu = walk.next(lu);
            lj = walk.first_tile();
          }
          then = look_up();
        }
        const int at = 16 * (int)(lx & 3);
        lives = (lives & ~(0xffffull << at)) | (unsigned long long)now.live << at;
      }
      if (now.live) {
        const __nv_bfloat16* from = lv ? p.v : p.k;
        if (!PAGED && KIND != kSegBlocks && lx < walk.prefix_tiles()) from = lv ? p.vp : p.kp;
        constexpr int CH = D / 8, RPP = 32 / (CH < 32 ? CH : 32);  // chunks a row, rows a pass
        const int c = lane % CH, r0 = lane / CH;
        const __nv_bfloat16* src = from + now.off + r0 * row_step + c * 8;
        const uint32_t dst = ring_s + ls * Gm::GRAN + r0 * Gm::ROWB;
        if (now.live == 0xffffu) {
#pragma unroll
          for (int r = 0; r < 16; r += RPP) {
            cp_async16(dst + r * Gm::ROWB + ((c ^ ((r + r0) & 7)) << 4), src, true);
            src += RPP * row_step;
          }
        } else {
#pragma unroll 1
          for (int r = 0; r < 16; r += RPP) {
            const bool is = (now.live >> (r + r0)) & 1;
            cp_async16(dst + r * Gm::ROWB + ((c ^ ((r + r0) & 7)) << 4), is ? src : from, is);
            src += RPP * row_step;
          }
        }
      }
      if (lv) {
        ++lx;
        now = then;
        ahead = false;
      }
      lv = !lv;
      ls = ls + 1 == NG ? 0 : ls + 1;
    }
    cp_async_commit();
  };

  int j = start;
  SegUnit u = u0;
#pragma unroll 1
  for (int s = 0; s < NG; ++s) issue();

  // column n of an MMA is the unit's row 8 nt + n; this lane's columns are 2 (lane % 4) and the next
  // values that are not finite, where not every row sees them: whether there are any in this unit, then 8 bits a
  // (row, element); and the tokens that each row sees
  uint32_t* odd_values = reinterpret_cast<uint32_t*>(smem + Gm::OFF_ODD);
  int* row_lims = reinterpret_cast<int*>(smem + Gm::OFF_ODD) + 1 + Gm::ROWS * D / 4;
  if constexpr (KIND == kSegEdges)
    for (int e = threadIdx.x; e < 1 + Gm::ROWS * D / 4; e += Gm::THREADS) odd_values[e] = 0u;

  uint32_t qb[NT][D / 16][2];
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];
  int lim[NT][2];
  int some_see = 0;  // tokens that every row sees which sees any
  bool fresh = true;
  int slot_at = 0;  // of the granule that is read next
  for (long long x = x0; x < x1; ++x) {
    if (fresh) {  // a new unit: its queries
      fresh = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        int token, g, unused;
        const bool is = seg_query<KIND>(p, walk.lens, u, 8 * nt + lane / 4, token, g, unused);
        const uint32_t* src =
            reinterpret_cast<const uint32_t*>(p.q + ((size_t)token * p.Hq + u.h * p.G + g) * D) + lane % 4;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qb[nt][kk][0] = is ? load_dependent(src + 8 * kk) : 0u;
          qb[nt][kk][1] = is ? load_dependent(src + 8 * kk + 4) : 0u;
          o[nt][kk][0] = o[nt][kk][1] = o[nt][kk][2] = o[nt][kk][3] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[nt][e] = kNegInf;
          l[nt][e] = 0.f;
          if (KIND == kSegEdges && !seg_query<KIND>(p, walk.lens, u, 8 * nt + 2 * (lane % 4) + e, token, g, lim[nt][e]))
            lim[nt][e] = 0x7fffffff;  // no row
        }
      }
      if constexpr (KIND == kSegEdges) {
        int seen = 0x7fffffff;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (lim[nt][e] > 0) seen = min(seen, lim[nt][e]);
        if (warp == 0 && lane < 4) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            row_lims[8 * nt + 2 * lane] = lim[nt][0];
            row_lims[8 * nt + 2 * lane + 1] = lim[nt][1];
          }
        }
        __syncthreads();
        some_see = __reduce_min_sync(0xffffffffu, seen);
      }
    }
    const bool last = j + 1 == walk.end_tile(u), join = last || x + 1 == x1;
    const uint32_t kst = ring_s + slot_at * Gm::GRAN;
    const int k_slot = slot_at;
    slot_at = slot_at + 1 == NG ? 0 : slot_at + 1;
    cp_async_wait<NG - 1>();
    __syncwarp();
    const uint32_t live = (uint32_t)(lives >> (16 * (int)(x & 3))) & 0xffffu;
    const int mrow = lane & 7, mi = lane >> 3;
    uint32_t pb[NT][2];
    const int g0 = (KIND != kSegBlocks && !u.prefix ? p.base & ~15 : 0) + j * kTile + warp * 16;  // the warp's first token
    if (live) {
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t a0, a1, a2, a3;  // tokens 0 .. 7 and 8 .. 15 of the first 8 elements, then of the second
        const int row = lane & 15, c = 2 * kk + (lane >> 4);
        ldsm_x4(kst + row * Gm::ROWB + ((c ^ mrow) << 4), a0, a1, a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(s[nt], a0, a1, a2, a3, qb[nt][kk][0], qb[nt][kk][1]);
      }
      const int t0 = g0 + lane / 4;
      float mx[NT][2];
      bool any = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            bool see = (live >> (lane / 4 + 8 * hf)) & 1;
            if (KIND == kSegEdges) see = see && t0 + 8 * hf < lim[nt][e];
            s[nt][2 * hf + e] = see ? s[nt][2 * hf + e] * p.scale_log2 : kNegInf;
          }
          float t = fmaxf(s[nt][e], s[nt][2 + e]);
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
          mx[nt][e] = t;
          any = any || t > m[nt][e] + 8.f;
        }
      if (__any_sync(0xffffffffu, any)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool raise = mx[nt][e] > m[nt][e] + 8.f;
            const float to = raise ? mx[nt][e] : m[nt][e];
            const float alpha = raise ? exp2_approx(m[nt][e] - to) : 1.f;  // 0 from -inf
            m[nt][e] = to;
            l[nt][e] *= alpha;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[nt][i][e] *= alpha;
              o[nt][i][2 + e] *= alpha;
            }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mu = m[nt][e] == kNegInf ? 0.f : m[nt][e];
          s[nt][e] = exp2_approx(s[nt][e] - mu);
          s[nt][2 + e] = exp2_approx(s[nt][2 + e] - mu);
          l[nt][e] += s[nt][e] + s[nt][2 + e];
        }
        // the weights go into the product as bf16 (2^-8 of each at most, as the output's own rounding)
        pb[nt][0] = transpose8x8(pack_bf16x2(s[nt][0], s[nt][1]));
        pb[nt][1] = transpose8x8(pack_bf16x2(s[nt][2], s[nt][3]));
      }
    }
    // the keys' place is free, unless the warps are joined now
    __syncwarp();
    if (!join) issue();
    const uint32_t vst = ring_s + slot_at * Gm::GRAN;
    const int v_slot = slot_at;
    slot_at = slot_at + 1 == NG ? 0 : slot_at + 1;
    if (join)
      cp_async_wait<NG - 2>();
    else
      cp_async_wait<NG - 1>();
    __syncwarp();
    if (KIND == kSegEdges && live && g0 + 16 > some_see) {
      // Tokens that some rows see and others do not: a weight of 0 times an infinity or NaN would reach the
      // others.  Such values leave the products, and the rows that see them are marked.
      uint32_t odd = 0u;  // an exponent of ones carries into the bit above it
#pragma unroll
      for (int c = 0; c < 16 * D / 8; c += 32) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(vst + (c + lane) * 16));
#pragma unroll
        for (int k = 0; k < 4; ++k) odd |= (w[k] & 0x7f807f80u) + 0x00800080u;
      }
      const bool any = __any_sync(0xffffffffu, odd & 0x80008000u);
#pragma unroll 1
      for (int c = lane; any && c < 16 * D / 8; c += 32) {
        const int t = c / (D / 8), d0 = ((c % (D / 8)) ^ (t & 7)) * 8;
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
          uint16_t* at = reinterpret_cast<uint16_t*>(smem + warp * Gm::WARP_BYTES + v_slot * Gm::GRAN + c * 16) + k;
          const uint32_t v = *at;
          if ((v & 0x7f80u) != 0x7f80u) continue;
          *at = 0;
          if (!((live >> t) & 1)) continue;
          odd_values[0] = 1u;
          const uint32_t mark = v & 0x7fu ? 4u : v >> 15 ? 2u : 1u;  // NaN, -inf, inf
          for (int n = 0; n < Gm::ROWS; ++n)
            if (g0 + t < row_lims[n]) atomicOr(&odd_values[1 + (n * D + d0 + k) / 4], mark << 8 * (k & 3));
        }
      }
      __syncwarp();
    }
    if (live) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t a0, a1, a2, a3;  // elements 0 .. 7 and 8 .. 15 of tokens 0 .. 7, then of 8 .. 15
        const int row = (mi >> 1) * 8 + mrow, c = 2 * i + (mi & 1);
        ldsm_x4_t(vst + row * Gm::ROWB + ((c ^ mrow) << 4), a0, a1, a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(o[nt][i], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
      }
    }
    __syncwarp();
    if (join) {
      // join the warps: each leaves 8 rows of its O in the places of the values (and the keys) that it has read
      float2* ml = reinterpret_cast<float2*>(smem + Gm::OFF_ML);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float* dst = reinterpret_cast<float*>(smem + warp * Gm::WARP_BYTES + (nt == 0 ? v_slot : k_slot) * Gm::GRAN);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = l[nt][e];
          t += __shfl_xor_sync(0xffffffffu, t, 4);
          t += __shfl_xor_sync(0xffffffffu, t, 8);
          t += __shfl_xor_sync(0xffffffffu, t, 16);
          const int n = 2 * (lane % 4) + e;
          if (lane < 4) ml[warp * Gm::ROWS + 8 * nt + n] = make_float2(m[nt][e], t);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const int d = 16 * i + lane / 4;
            dst[n * D + (d ^ ((lane % 4) << 3))] = o[nt][i][e];
            dst[n * D + ((d + 8) ^ ((lane % 4) << 3))] = o[nt][i][2 + e];
          }
        }
      }
      __syncthreads();
      const bool whole = KIND == kSegBlocks && p.cluster == 1;
      const size_t slot = (size_t)u.id + blockIdx.x;
      float2* res_ml = reinterpret_cast<float2*>(smem + Gm::OFF_RES);  // blocks shared by a cluster
      float* res_o = reinterpret_cast<float*>(smem + Gm::OFF_RES + Gm::ROWS * 8);
      // each row's factors of the warps' O, and where it goes
      FoldRow* fold = reinterpret_cast<FoldRow*>(smem + Gm::OFF_FOLD);
      if (threadIdx.x < Gm::ROWS) {
        const int r = threadIdx.x;
        int token, g, unused;
        float mw[Gm::WARPS], lw[Gm::WARPS], M = kNegInf, L = 0.f;
#pragma unroll
        for (int w = 0; w < Gm::WARPS; ++w) {
          const float2 y = ml[w * Gm::ROWS + r];
          mw[w] = y.x;
          lw[w] = y.y;
          M = fmaxf(M, y.x);
        }
        FoldRow f;
#pragma unroll
        for (int w = 0; w < Gm::WARPS; ++w) {
          // l = 0: saw nothing (scores of NaN alone leave m at -inf and l at NaN)
          f.f[w] = lw[w] == 0.f ? 0.f : mw[w] == kNegInf ? 1.f : exp2_approx(mw[w] - M);
          L += f.f[w] * lw[w];
        }
        f.out = seg_query<KIND>(p, walk.lens, u, r, token, g, unused) ? ((long long)token * p.Hq + u.h * p.G + g) * D : -1;
        if (whole) {
          const float inv = L == 0.f ? 0.f : 1.f / L;  // a row that saw nothing is zeros
#pragma unroll
          for (int w = 0; w < Gm::WARPS; ++w) f.f[w] *= inv;
        } else if (KIND == kSegBlocks) {
          res_ml[r] = make_float2(M, L);
        } else if (f.out >= 0) {
          p.part_ml[slot * Gm::ROWS + r] = make_float2(M, L);
        }
        fold[r] = f;
      }
      __syncthreads();
#pragma unroll 2
      for (int e = threadIdx.x; e < Gm::ROWS * (D / 4); e += Gm::THREADS) {
        const int r = e / (D / 4), n = r % 8, c = (e % (D / 4)) * 4;
        const FoldRow f = fold[r];
        if (f.out < 0) break;
        const uint8_t* from = smem + (r < 8 ? v_slot : k_slot) * Gm::GRAN;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < Gm::WARPS; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(from + w * Gm::WARP_BYTES) +
                                                            n * D + (c ^ ((n >> 1) << 3)));
          if (f.f[w] == 0.f) continue;
          a.x += f.f[w] * y.x;
          a.y += f.f[w] * y.y;
          a.z += f.f[w] * y.z;
          a.w += f.f[w] * y.w;
        }
        if (KIND == kSegEdges && odd_values[0]) {
          const uint32_t marks = odd_values[1 + (r * D + c) / 4];
          a.x += odd_value(marks);
          a.y += odd_value(marks >> 8);
          a.z += odd_value(marks >> 16);
          a.w += odd_value(marks >> 24);
        }
        if (whole)
          *reinterpret_cast<uint2*>(p.out + f.out + c) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
        else if (KIND == kSegBlocks)
          *reinterpret_cast<float4*>(res_o + r * D + c) = a;
        else
          *reinterpret_cast<float4*>(p.part_o + (slot * Gm::ROWS + r) * D + c) = a;
      }
      if (KIND == kSegBlocks && p.cluster > 1) {
        // the cluster's CTAs join a share of the rows' elements each
        cluster_sync();
        const int rank = blockIdx.x % p.cluster, all = Gm::ROWS * (D / 4);
        for (int e = all * rank / p.cluster + threadIdx.x; e < all * (rank + 1) / p.cluster; e += Gm::THREADS) {
          const int r = e / (D / 4), c = (e % (D / 4)) * 4;
          const long long to = fold[r].out;
          if (to < 0) break;
          float2 y[kSegCluster];
          float M = kNegInf, L = 0.f;
#pragma unroll
          for (int k = 0; k < kSegCluster; ++k) {
            y[k] = k < p.cluster ? load_at<float2>(smem_u32(res_ml + r), k) : make_float2(kNegInf, 0.f);
            M = fmaxf(M, y[k].x);
          }
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < kSegCluster; ++k) {
            if (y[k].y == 0.f) continue;
            const float w = y[k].x == kNegInf ? 1.f : exp2_approx(y[k].x - M);
            const float4 z = load_at<float4>(smem_u32(res_o + r * D + c), k);
            L += w * y[k].y;
            a.x += w * z.x;
            a.y += w * z.y;
            a.z += w * z.z;
            a.w += w * z.w;
          }
          const float inv = L == 0.f ? 0.f : 1.f / L;  // a row that saw nothing is zeros
          *reinterpret_cast<uint2*>(p.out + to + c) =
              make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
        }
        cluster_sync();  // no CTA writes its own again, or leaves, before all have read it
      } else {
        __syncthreads();
      }
      if (KIND == kSegEdges && odd_values[0]) {
        __syncthreads();
        for (int e = threadIdx.x; e < 1 + Gm::ROWS * D / 4; e += Gm::THREADS) odd_values[e] = 0u;
        __syncthreads();
      }
      issue();
    }
    issue();
    ++j;
    if (last && x + 1 < x1) {
      u = walk.next(u);
      j = walk.first_tile();
      fresh = true;
    }
  }
  cp_async_wait<0>();
  if (p.beside) pdl_wait_primary();
}

// One row's partials joined by a warp: pieces [0, count), at(k, ml, o) gives the places of its
// (m, l) and O.  Each lane ends with columns 4 lane + 128 k .. + 3 of O / l (D = 64: 2 lane, + 1).
template <int D>
struct SegRow {
  static constexpr int N = D / 32;
  float a[N];
  float m, l;
  __device__ __forceinline__ SegRow() : m(kNegInf), l(0.f) {
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = 0.f;
  }
  template <typename F>
  __device__ __forceinline__ void add(int count, F at) {
    const int lane = threadIdx.x & 31;
    for (int k0 = 0; k0 < count; k0 += 32) {
      const float2* ml = nullptr;
      const float* o = nullptr;
      if (k0 + lane < count) at(k0 + lane, ml, o);
      const float2 mine = ml ? __ldcg(ml) : make_float2(kNegInf, 0.f);
      const int here = min(32, count - k0);
      const unsigned long long from = reinterpret_cast<unsigned long long>(o);
      // the loads do not wait for the weights: U pieces at a time
      constexpr int U = 8;
      float w = 0.f, old = 1.f;
      for (int i0 = 0; i0 < here; i0 += U) {
        float y[U][N];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const float* src = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, from, i0 + i & 31));
#pragma unroll
          for (int c = 0; c < N; ++c) y[i][c] = 0.f;
          if (i0 + i < here) {
            if constexpr (D == 64) {
              const float2 v = __ldcg(reinterpret_cast<const float2*>(src) + lane);
              y[i][0] = v.x;
              y[i][1] = v.y;
            } else {
#pragma unroll
              for (int c = 0; c < D / 128; ++c) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(src) + lane + 32 * c);
                y[i][4 * c] = v.x;
                y[i][4 * c + 1] = v.y;
                y[i][4 * c + 2] = v.z;
                y[i][4 * c + 3] = v.w;
              }
            }
          }
        }
        if (i0 == 0) {
          float M = mine.x;
#pragma unroll
          for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
          M = fmaxf(M, m);
          const float mu = M == kNegInf ? 0.f : M;
          const bool empty = mine.y == 0.f;
          old = m == kNegInf ? 1.f : exp2_approx(m - mu);  // nothing yet, or NaN
          w = empty ? 0.f : mine.x == kNegInf ? 1.f : exp2_approx(mine.x - mu);
          m = M;
          float s = empty ? 0.f : w * mine.y;
#pragma unroll
          for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
          l = l * old + s;
#pragma unroll
          for (int i = 0; i < N; ++i) a[i] *= old;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const float f = __shfl_sync(0xffffffffu, w, i0 + i & 31);
          const bool none = __shfl_sync(0xffffffffu, mine.y, i0 + i & 31) == 0.f;  // its O may be anything
          if (none || i0 + i >= here) continue;
#pragma unroll
          for (int c = 0; c < N; ++c) a[c] += f * y[i][c];
        }
      }
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* dst) const {
    const int lane = threadIdx.x & 31;
    const bool none = l == 0.f;  // a row that saw nothing is zeros
    const float f = none ? 0.f : 1.f / l;
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = none ? 0u : pack_bf16x2(a[2 * i] * f, a[2 * i + 1] * f);
    if constexpr (D == 64) {
      reinterpret_cast<uint32_t*>(dst)[lane] = w[0];
    } else {
#pragma unroll
      for (int c = 0; c < D / 128; ++c) reinterpret_cast<uint2*>(dst)[lane + 32 * c] = make_uint2(w[2 * c], w[2 * c + 1]);
    }
  }
};

constexpr int kMergeThreads = 256;

// On the tensor cores a value of the prefix meets every row, with a weight of 0 where the row's sequence ends before it; if it
// is not finite, that is NaN.  A row that sees a part of the prefix alone is computed here by itself, by its warp: 32 tokens
// at a time, a lane the score of one and then its columns of the sum; 0.2 us a token.  (Not inlined: it is rare.)
template <int D>
__device__ __noinline__ void seg_row_of_prefix(const SegParams& p, long long row) {
  const int lane = threadIdx.x & 31, row_step = p.Hkv * D;
  const int hq = (int)(row % p.Hq), token = (int)(row / p.Hq), h = hq / p.G, b = token / p.n;
  const int seen = seg_len(p.seq_lens, b, p.cap) - p.n + 1 + (token - b * p.n);
  if (seen <= 0 || seen >= p.base) return;
  SegRow<D> acc;
  const __nv_bfloat16 *keys = p.prefix_table ? p.k : p.kp, *values = p.prefix_table ? p.v : p.vp;
  const uint4* q = reinterpret_cast<const uint4*>(p.q + ((size_t)token * p.Hq + hq) * D);
#pragma unroll 1
  for (int t0 = 0; t0 < seen; t0 += 32) {
    const int t = t0 + lane;
    long long at = t;
    float s = kNegInf;
    if (t < seen) {
      if (p.prefix_table) {
        const int col = t / p.page_size, page = load_dependent(p.prefix_table + col);
        at = ((unsigned)page < (unsigned)p.num_pages ? (long long)page : 0ll) * p.page_size + (t - col * p.page_size);
      }
      const uint4* k = reinterpret_cast<const uint4*>(keys + at * row_step + h * D);
      s = 0.f;
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = load_dependent(q + c), y = load_dependent(k + c);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s = fmaf(bf16lo_to_f32(xs[i]), bf16lo_to_f32(ys[i]), s);
          s = fmaf(bf16hi_to_f32(xs[i]), bf16hi_to_f32(ys[i]), s);
        }
      }
      s *= p.scale_log2;
    }
    float top = fmaxf(acc.m, s);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float mu = top == kNegInf ? 0.f : top, old = acc.m == kNegInf ? 1.f : exp2_approx(acc.m - mu);
    const float w = exp2_approx(s - mu);
    float sum = w;
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    acc.m = top;
    acc.l = acc.l * old + sum;
#pragma unroll
    for (int c = 0; c < SegRow<D>::N; ++c) acc.a[c] *= old;
#pragma unroll 8
    for (int i = 0; i < min(32, seen - t0); ++i) {
      const float f = __shfl_sync(0xffffffffu, w, i);
      const __nv_bfloat16* v = values + __shfl_sync(0xffffffffu, at, i) * row_step + h * D;
#pragma unroll
      for (int c = 0; c < SegRow<D>::N / 2; ++c) {
        // columns as SegRow has them
        const uint32_t y = load_dependent(reinterpret_cast<const uint32_t*>(v) + (D == 64 ? lane : 2 * lane + 64 * (c / 2) + c % 2));
        acc.a[2 * c] += f * bf16lo_to_f32(y);
        acc.a[2 * c + 1] += f * bf16hi_to_f32(y);
      }
    }
  }
  acc.store(p.out + row * D);
}

// Joins the prefix's and the rests' partials: a warp a row of the output, the loads of 8 pieces in flight.  33 MB for 64
// x 64 heads of 128: 8 us behind the rests' kernel.  The lengths are read
// before the wait: the kernels that wrote them were done before seg_kernel, and prefix_tc_kernel
// before it, let anything start.
template <int D>
__global__ void __launch_bounds__(kMergeThreads, D == 256 ? 2 : 4) seg_merge_prefix_kernel(const __grid_constant__ SegParams p) {
  const long long row = (long long)blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);
  if (row >= (long long)p.B * p.n * p.Hq) {
    pdl_wait_primary();
    return;
  }
  const int hq = (int)(row % p.Hq), token = (int)(row / p.Hq);
  const int b = token / p.n, i = token - b * p.n, h = hq / p.G, g = hq - h * p.G;
  const SegSums sums = seg_sums(p.seq_lens, p.B, p.cap, p.base & ~15, b);
  const long long tp = p.rt_prefix ? (p.base + kTile - 1) / kTile : 0, wp = (long long)p.Hkv * p.rt_prefix * tp;
  const long long W = wp + sums.all * p.Hkv * p.rt;
  const int used = seg_used(W, p.ctas);
  // the prefix's pieces: parts of prefix_tc_kernel, or of the unit of seg_kernel with its row
  const int head = token * p.G + g;  // among the rows of the head
  int na = p.slabs, id0 = 0, c0 = 0;
  if (!p.slabs && p.rt_prefix && tp > 0) {
    id0 = h * p.rt_prefix + head / p.ru;
    c0 = seg_owner(W, used, id0 * tp);
    na = seg_owner(W, used, (id0 + 1) * tp - 1) - c0 + 1;
  }
  // the rest's
  const int rr = i * p.G + g, r = rr / p.ru, t = seg_tiles(seg_len(p.seq_lens, b, p.cap), p.cap, p.base & ~15);
  const long long a1 = wp + sums.before * p.Hkv * p.rt + (long long)(h * p.rt + r) * t;
  const int id1 = p.Hkv * p.rt_prefix + (b * p.Hkv + h) * p.rt + r;
  const int c1 = t ? seg_owner(W, used, a1) : 0, nb = t ? seg_owner(W, used, a1 + t - 1) - c1 + 1 : 0;
  pdl_wait_primary();
  SegRow<D> acc;
  acc.add(na + nb, [&](int k, const float2*& ml, const float*& o) {
    if (k < na && p.slabs) {
      const long long at = ((long long)k * p.Hkv + h) * ((long long)p.B * p.n * p.G) + head;
      ml = p.tc_ml + at;
      o = p.tc_o + at * D;
    } else {
      const long long at = k < na ? ((long long)id0 + c0 + k) * p.ru + head % p.ru
                                  : ((long long)id1 + c1 + k - na) * p.ru + rr % p.ru;
      ml = p.part_ml + at;
      o = p.part_o + at * D;
    }
  });
  acc.store(p.out + row * D);
  if (p.slabs) {
    bool odd = false;
#pragma unroll
    for (int c = 0; c < SegRow<D>::N; ++c) odd = odd || !(acc.a[c] - acc.a[c] == 0.f);
    if (__any_sync(0xffffffffu, odd)) seg_row_of_prefix<D>(p, row);
  }
}

}  // namespace da
