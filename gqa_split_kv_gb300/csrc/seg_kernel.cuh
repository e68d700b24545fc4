// Attention of query rows over lists of cached tokens, for few rows a KV head: the tokens
// [base, L) of a sequence, the first base tokens that a batch shares, or the blocks that
// were selected for a query.  16 rows at a time on the warp-level MMA, as the tokens' bytes
// bound it: a CTA reads each key and value once for its 16 rows.
//
// The 4 warps of a CTA take 16 tokens each of every tile of 64 and run on their own, with
// no barrier between them: a warp looks up where its tokens lie one tile ahead, copies
// their rows into its own ring (cp.async; rows that do not exist are zeros there), and keeps
// a running maximum m, sum l and output O of its tokens,
//     O = sum_t 2^(s_t - m) v_t,   l = sum_t 2^(s_t - m),   s_t = scale log2(e) <q, k_t>.
// Where a unit ends (seg_plan.cuh) the warps' four (m, l, O) are joined through shared memory
// and written as one partial, or as the output where the CTA had the whole unit.  m is only
// raised when a score passes it by more than 8; it cancels in O / l.
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

constexpr int kSegLens = 1024;  // lengths that a CTA copies to its shared memory

enum SegKind { kSegRange = 0, kSegBlocks = 1 };

struct SegParams {
  const __nv_bfloat16* q;      // [B, n, Hq, D]
  const __nv_bfloat16 *k, *v;  // contiguous [B, ctx, Hkv, D] (token t in row t - base), or pools
  const __nv_bfloat16 *kp, *vp;  // the shared prefix's cache, contiguous: [base, Hkv, D]
  const int* seq_lens;         // prefix included; null: cap
  const int *page_table, *prefix_table;
  const int* blocks;           // [B, n, Hkv, pick]
  __nv_bfloat16* out;          // like q
  float* part_o;               // [slots][16][D]; slots: seg_plan.cuh's, of blocks 2 c + 1 for the piece of CTA c that
                               // starts a unit, 2 c for one that goes on with it
  float2* part_ml;             // [slots][16]: m, l
  const float* tc_o;           // [slabs][Hkv][B n G][D]: the prefix's partials, where another kernel made them
  const float2* tc_ml;
  int slabs;
  int B, n, Hq, Hkv, G;
  int base;                    // tokens of the shared prefix
  int cap;                     // longest sequence
  int ctx;
  int page_size, max_pages, num_pages;
  int block, pick;
  int rt, rt_prefix;           // tiles of 16 query rows a sequence's KV head, and of the prefix's (0: none here)
  int ctas;                    // of seg_kernel: the plan's n
  int beside;                  // the kernel before is the prefix's: seg_kernel runs beside it and waits for it at its end
  float scale_log2;
};

// A row where a unit's warps are joined: their factors, and its place in the output (-1: no row).
struct FoldRow {
  float f[4];
  long long out;
};

template <int D>
struct SegGeo {
  static constexpr int WARPS = 4, THREADS = 32 * WARPS;
  static constexpr int ROWB = 2 * D;            // a row of K or V
  static constexpr int STAGE = 2 * 16 * ROWB;   // 16 tokens of both; also 16 rows of O in fp32
  static constexpr int NSTAGE = D == 64 ? 6 : 3;
  static constexpr int WARP_BYTES = NSTAGE * STAGE;
  static constexpr int OFF_ML = WARPS * WARP_BYTES;
  static constexpr int OFF_FOLD = OFF_ML + WARPS * 16 * 8;
  static constexpr int OFF_MASK = OFF_FOLD + 16 * (int)sizeof(FoldRow);
  static constexpr int OFF_LENS = OFF_MASK + WARPS * NSTAGE * 4;
  static constexpr int SMEM = OFF_LENS + kSegLens * 4;
  static constexpr int PER_SM = D == 256 ? 1 : 2;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
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

// A unit: 16 query rows (from row 16 r of its rows) of KV head h, and its tokens.
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
  int tp;         // tiles of a prefix unit
  int used;       // CTAs that have some

  __device__ __forceinline__ SegWalk(const SegParams& p_, const int* lens_) : p(p_), lens(lens_), all(0), tp(0), used(0) {
    if constexpr (KIND == kSegBlocks) {
      tp = (p.pick * p.block + kTile - 1) / kTile;
      all = (long long)p.B * p.n * p.Hkv * p.rt * tp;
    } else {
      tp = p.rt_prefix ? (p.base + kTile - 1) / kTile : 0;
      all = seg_sums(lens, p.B, p.cap, p.base, 0).all * p.Hkv * p.rt + prefix_tiles();
    }
    used = seg_used(all, p.ctas);
  }
  // The tiles [x0, x1) of a CTA; none past those used.
  __device__ __forceinline__ bool range(int c, long long& x0, long long& x1) const {
    if (c >= used) return false;
    x0 = seg_start(all, used, c);
    x1 = seg_start(all, used, c + 1);
    return true;
  }
  __device__ __forceinline__ long long prefix_tiles() const { return (long long)p.Hkv * p.rt_prefix * tp; }

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
    u.tiles = seg_tiles(u.end, p.cap, p.base);
    u.id = p.Hkv * p.rt_prefix + (b * p.Hkv + h) * p.rt + r;
    return u;
  }
  // The unit of tile x (x < all), j: the tile's place in it.  The warp executes it.
  __device__ __forceinline__ SegUnit at(long long x, int& j) const {
    if constexpr (KIND == kSegBlocks) {
      const int id = (int)seg_div(x, tp);
      j = (int)(x - (long long)id * tp);
      return blocks_unit(id);
    } else {
      const long long wp = prefix_tiles();
      if (x < wp) {
        const int id = (int)seg_div(x, tp);
        j = (int)(x - (long long)id * tp);
        return prefix_unit(id);
      }
      x -= wp;
      const int hr = p.Hkv * p.rt;
      const SegAt f = seg_find(lens, p.B, p.cap, p.base, seg_div(x, hr));
      const int tb = seg_tiles(seg_len(lens, f.b, p.cap), p.cap, p.base);
      const long long in = x - f.start * hr;
      const int w = (int)seg_div(in, tb);
      j = (int)(in - (long long)w * tb);
      return range_unit(f.b, w / p.rt, w % p.rt);
    }
  }
  // The next unit that has tiles; there is one.
  __device__ __forceinline__ SegUnit next(const SegUnit& u) const {
    if constexpr (KIND == kSegBlocks) {
      return blocks_unit(u.id + 1);
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

// Element offset of a token's row of head h in the cache (or the prefix's), -1 where there
// is none.  A page outside the pool is flagged and page 0 read instead.
template <int D, bool PAGED, int KIND>
__device__ __forceinline__ long long seg_row(const SegParams& p, const SegUnit& u, int at) {
  int t;  // the token
  if constexpr (KIND == kSegBlocks) {
    const int e = at / p.block;
    if (e >= p.pick) return -1;
    const int id = load_dependent(p.blocks + (((size_t)u.b * p.n + u.i) * p.Hkv + u.h) * p.pick + e);
    if (id < 0 || id > (u.end - 1) / p.block) return -1;
    t = id * p.block + (at - e * p.block);
  } else {
    t = at + (u.prefix ? 0 : p.base);
  }
  if (t >= u.end) return -1;
  if constexpr (PAGED) {
    const int col = t / p.page_size;
    int page = load_dependent(u.prefix ? p.prefix_table + col : p.page_table + (size_t)u.b * p.max_pages + col);
    if ((unsigned)page >= (unsigned)p.num_pages) {
      atomicOr(&g_error_word, 4u);
      page = 0;
    }
    return (((long long)page * p.page_size + (t - col * p.page_size)) * p.Hkv + u.h) * D;
  } else {
    const long long row = u.prefix ? t : (long long)u.b * p.ctx + (t - p.base);
    return (row * p.Hkv + u.h) * D;
  }
}

// Row rr of a unit: its query token (over the batch), head in the group, and how many tokens
// it sees; false past the unit's rows.
template <int KIND>
__device__ __forceinline__ bool seg_query(const SegParams& p, const int* lens, const SegUnit& u, int rr, int& token, int& g,
                                          int& lim) {
  const int row = u.r * 16 + rr;
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

template <int D, bool PAGED, int KIND>
__global__ void __launch_bounds__(SegGeo<D>::THREADS, SegGeo<D>::PER_SM) seg_kernel(const __grid_constant__ SegParams p) {
  using Gm = SegGeo<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * Gm::WARP_BYTES;
  const uint32_t ring_s = smem_u32(ring);
  volatile uint32_t* masks = reinterpret_cast<volatile uint32_t*>(smem + Gm::OFF_MASK) + warp * Gm::NSTAGE;

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

  // the load side: where the rows of the next copy lie (lanes 0 .. 15), and of the one after it;
  // lu and lj are the unit and tile of the latter
  int lj;
  SegUnit lu = walk.at(x0, lj);
  const SegUnit u0 = lu;
  const int start = lj;
  long long lx = x0;  // the next copy's tile
  auto look_up = [&]() {
    return lane < 16 ? seg_row<D, PAGED, KIND>(p, lu, lj * kTile + warp * 16 + lane) : -1ll;
  };
  auto advance = [&](long long x) {  // to tile x, the one after lu's and lj's; none past the last
    if (x >= x1) return;
    if (++lj == lu.tiles) {
      lu = walk.next(lu);
      lj = 0;
    }
  };
  long long off = look_up(), off_next = -1;
  advance(x0 + 1);
  if (x0 + 1 < x1) off_next = look_up();
  auto issue = [&](int stage) {
    if (lx < x1) {
      const uint32_t live = __ballot_sync(0xffffffffu, off >= 0);
      if (lane == 0) masks[stage] = live;
      if (live) {
        const uint32_t dst = ring_s + stage * Gm::STAGE;
        const __nv_bfloat16 *kb = p.k, *vb = p.v;
        if (!PAGED && KIND == kSegRange && lx < walk.prefix_tiles()) {
          kb = p.kp;
          vb = p.vp;
        }
        constexpr int CH = D / 8, RPP = 32 / (CH < 32 ? CH : 32);  // chunks a row, rows a pass
        const int c = lane % CH, r0 = lane / CH;
#pragma unroll
        for (int r = 0; r < 16; r += RPP) {
          const int row = r + r0;
          const long long o = __shfl_sync(0xffffffffu, off, row);
          const size_t e = (size_t)(o < 0 ? 0 : o) + c * 8;
          const uint32_t d = dst + row * Gm::ROWB + ((c ^ (row & 7)) << 4);
          cp_async16(d, kb + e, o >= 0);
          cp_async16(d + 16 * Gm::ROWB, vb + e, o >= 0);
        }
      }
      ++lx;
      off = off_next;
      advance(lx + 1);
      if (lx + 1 < x1) off_next = look_up();
    }
    cp_async_commit();
  };

  int j = start;
  SegUnit u = u0;
#pragma unroll 1
  for (int s = 0; s < Gm::NSTAGE; ++s) issue(s);

  uint32_t qa[D / 16][4];
  float o[D / 8][4];
  float m[2], l[2];
  int lim[2];
  int j0 = j;
  bool fresh = true;
  int stage = 0;
  for (long long x = x0; x < x1; ++x) {
    if (fresh) {  // a new unit: its queries
      fresh = false;
      j0 = j;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        int token, g;
        const bool is = seg_query<KIND>(p, walk.lens, u, lane / 4 + 8 * hf, token, g, lim[hf]);
        const uint32_t* src =
            reinterpret_cast<const uint32_t*>(p.q + ((size_t)token * p.Hq + u.h * p.G + g) * D) + lane % 4;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qa[kk][hf] = is ? load_dependent(src + 8 * kk) : 0u;
          qa[kk][2 + hf] = is ? load_dependent(src + 8 * kk + 4) : 0u;
        }
        m[hf] = kNegInf;
        l[hf] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
    cp_async_wait<Gm::NSTAGE - 1>();
    __syncwarp();
    const uint32_t live = masks[stage];
    if (live) {
      const uint32_t kst = ring_s + stage * Gm::STAGE, vst = kst + 16 * Gm::ROWB;
      const int mrow = lane & 7, mi = lane >> 3;
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t r0, r1, r2, r3;
        const int row = (mi >> 1) * 8 + mrow, c = 2 * kk + (mi & 1);
        ldsm_x4(kst + row * Gm::ROWB + ((c ^ mrow) << 4), r0, r1, r2, r3);
        mma_bf16_16816(s[0], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], r0, r1);
        mma_bf16_16816(s[1], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], r2, r3);
      }
      const int t0 = (KIND == kSegRange && !u.prefix ? p.base : 0) + j * kTile + warp * 16;
      float mx[2] = {kNegInf, kNegInf};
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = nt * 8 + 2 * (lane % 4) + (e & 1);
          bool see = (live >> col) & 1;
          if (KIND == kSegRange) see = see && t0 + col < lim[e >> 1];
          s[nt][e] = see ? s[nt][e] * p.scale_log2 : kNegInf;
          mx[e >> 1] = fmaxf(mx[e >> 1], s[nt][e]);
        }
      float mu[2];
      bool raise[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 1));
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 2));
        raise[hf] = mx[hf] > m[hf] + 8.f;
      }
      if (__any_sync(0xffffffffu, raise[0] || raise[1])) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float to = raise[hf] ? mx[hf] : m[hf];
          const float alpha = raise[hf] ? exp2_approx(m[hf] - to) : 1.f;  // 0 from -inf
          m[hf] = to;
          l[hf] *= alpha;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[i][2 * hf] *= alpha;
            o[i][2 * hf + 1] *= alpha;
          }
        }
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        mu[hf] = m[hf] == kNegInf ? 0.f : m[hf];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          s[nt][2 * hf] = exp2_approx(s[nt][2 * hf] - mu[hf]);
          s[nt][2 * hf + 1] = exp2_approx(s[nt][2 * hf + 1] - mu[hf]);
          l[hf] += s[nt][2 * hf] + s[nt][2 * hf + 1];
        }
      }
      // the weights go into the product as bf16 (2^-9 of each, against the output's own 2^-9)
      const uint32_t a0 = pack_bf16x2(s[0][0], s[0][1]), a1 = pack_bf16x2(s[0][2], s[0][3]),
                     a2 = pack_bf16x2(s[1][0], s[1][1]), a3 = pack_bf16x2(s[1][2], s[1][3]);
#pragma unroll
      for (int nn = 0; nn < D / 16; ++nn) {
        uint32_t r0, r1, r2, r3;
        const int row = (mi & 1) * 8 + mrow, c = 2 * nn + (mi >> 1);
        ldsm_x4_t(vst + row * Gm::ROWB + ((c ^ mrow) << 4), r0, r1, r2, r3);
        mma_bf16_16816(o[2 * nn], a0, a1, a2, a3, r0, r1);
        mma_bf16_16816(o[2 * nn + 1], a0, a1, a2, a3, r2, r3);
      }
    }
    const bool last = j + 1 == u.tiles;
    if (last || x + 1 == x1) {
      // join the warps: each leaves its O in the ring slot that it has just read
      float2* ml = reinterpret_cast<float2*>(smem + Gm::OFF_ML);
      __syncwarp();
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 1);
        l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 2);
        const int r = lane / 4 + 8 * hf;
        if (lane % 4 == 0) ml[warp * 16 + r] = make_float2(m[hf], l[hf]);
        float* dst = reinterpret_cast<float*>(ring + stage * Gm::STAGE) + r * D;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<float2*>(dst + ((8 * i + 2 * (lane % 4)) ^ ((r & 3) << 3))) =
              make_float2(o[i][2 * hf], o[i][2 * hf + 1]);
      }
      __syncthreads();
      const bool whole = KIND == kSegBlocks && last && j0 == 0;
      const size_t slot = KIND == kSegBlocks ? 2 * (size_t)blockIdx.x + (j0 == 0) : (size_t)u.id + blockIdx.x;
      // each row's factors of the warps' O, and where it goes
      FoldRow* fold = reinterpret_cast<FoldRow*>(smem + Gm::OFF_FOLD);
      if (threadIdx.x < 16) {
        const int r = threadIdx.x;
        int token, g, unused;
        float mw[Gm::WARPS], lw[Gm::WARPS], M = kNegInf, L = 0.f;
#pragma unroll
        for (int w = 0; w < Gm::WARPS; ++w) {
          const float2 y = ml[w * 16 + r];
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
        } else if (f.out >= 0) {
          p.part_ml[slot * 16 + r] = make_float2(M, L);
        }
        fold[r] = f;
      }
      __syncthreads();
#pragma unroll 4
      for (int e = threadIdx.x; e < 16 * (D / 4); e += Gm::THREADS) {
        const int r = e / (D / 4), c = (e % (D / 4)) * 4;
        const FoldRow f = fold[r];
        if (f.out < 0) break;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < Gm::WARPS; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(
              reinterpret_cast<const float*>(smem + w * Gm::WARP_BYTES + stage * Gm::STAGE) + r * D + (c ^ ((r & 3) << 3)));
          if (f.f[w] == 0.f) continue;
          a.x += f.f[w] * y.x;
          a.y += f.f[w] * y.y;
          a.z += f.f[w] * y.z;
          a.w += f.f[w] * y.w;
        }
        if (whole)
          *reinterpret_cast<uint2*>(p.out + f.out + c) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
        else
          *reinterpret_cast<float4*>(p.part_o + (slot * 16 + r) * D + c) = a;
      }
      __syncthreads();
    }
    issue(stage);
    stage = stage + 1 == Gm::NSTAGE ? 0 : stage + 1;
    ++j;
    if (last && x + 1 < x1) {
      u = walk.next(u);
      j = 0;
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

// Joins the prefix's and the rests' partials: a warp a row of the output.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) seg_merge_prefix_kernel(const __grid_constant__ SegParams p) {
  pdl_wait_primary();
  const long long row = (long long)blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);
  if (row >= (long long)p.B * p.n * p.Hq) return;
  const int hq = (int)(row % p.Hq), token = (int)(row / p.Hq);
  const int b = token / p.n, i = token - b * p.n, h = hq / p.G, g = hq - h * p.G;
  const SegSums sums = seg_sums(p.seq_lens, p.B, p.cap, p.base, b);
  const long long tp = p.rt_prefix ? (p.base + kTile - 1) / kTile : 0, wp = (long long)p.Hkv * p.rt_prefix * tp;
  const long long W = wp + sums.all * p.Hkv * p.rt;
  const int used = seg_used(W, p.ctas);
  // the prefix's pieces: parts of prefix_tc_kernel, or of the unit of seg_kernel with its row
  const int head = token * p.G + g;  // among the rows of the head
  int na = p.slabs, id0 = 0, c0 = 0;
  if (!p.slabs && p.rt_prefix && tp > 0) {
    id0 = h * p.rt_prefix + head / 16;
    c0 = seg_owner(W, used, id0 * tp);
    na = seg_owner(W, used, (id0 + 1) * tp - 1) - c0 + 1;
  }
  // the rest's
  const int rr = i * p.G + g, r = rr / 16, t = seg_tiles(seg_len(p.seq_lens, b, p.cap), p.cap, p.base);
  const long long a1 = wp + sums.before * p.Hkv * p.rt + (long long)(h * p.rt + r) * t;
  const int id1 = p.Hkv * p.rt_prefix + (b * p.Hkv + h) * p.rt + r;
  const int c1 = t ? seg_owner(W, used, a1) : 0, nb = t ? seg_owner(W, used, a1 + t - 1) - c1 + 1 : 0;
  SegRow<D> acc;
  acc.add(na + nb, [&](int k, const float2*& ml, const float*& o) {
    if (k < na && p.slabs) {
      const long long at = ((long long)k * p.Hkv + h) * ((long long)p.B * p.n * p.G) + head;
      ml = p.tc_ml + at;
      o = p.tc_o + at * D;
    } else {
      const long long at = k < na ? ((long long)id0 + c0 + k) * 16 + head % 16 : ((long long)id1 + c1 + k - na) * 16 + rr % 16;
      ml = p.part_ml + at;
      o = p.part_o + at * D;
    }
  });
  acc.store(p.out + row * D);
}

// Joins the partials of the blocks units that were cut: CTA c looks at the start of CTA c + 1's
// tiles, and joins that unit if it is cut there first.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) seg_merge_blocks_kernel(const __grid_constant__ SegParams p) {
  pdl_wait_primary();
  const long long tp = (p.pick * p.block + kTile - 1) / kTile, W = (long long)p.B * p.n * p.Hkv * p.rt * tp;
  const long long x = seg_start(W, p.ctas, blockIdx.x + 1), id = seg_div(x, tp);
  if (x >= W || x == id * tp || seg_start(W, p.ctas, blockIdx.x) > id * tp) return;
  const int c0 = blockIdx.x, c1 = seg_owner(W, p.ctas, (id + 1) * tp - 1);
  const int r0 = (int)(id % p.rt) * 16, h = (int)(id / p.rt % p.Hkv);
  const long long token = id / p.rt / p.Hkv;
  for (int r = threadIdx.x >> 5; r < 16 && r0 + r < p.G; r += kMergeThreads / 32) {
    SegRow<D> acc;
    acc.add(c1 - c0 + 1, [&](int k, const float2*& ml, const float*& o) {
      const long long at = (2ll * (c0 + k) + (k == 0)) * 16 + r;
      ml = p.part_ml + at;
      o = p.part_o + at * D;
    });
    acc.store(p.out + (token * p.Hq + h * p.G + r0 + r) * D);
  }
}

}  // namespace da
