// The attention weight that new tokens give each cached token, summed over them and over the
// heads of a group.  A softmax needs its whole row's maximum and sum before the first weight
// is known, so there are two kernels:
//
// up to 16 rows (decode):
//   weights_score_kernel   reads every key once (warp-level MMA), writes the scores (4 bytes a row and token, a
//                          sixty-fourth of a 128-wide bf16 key a row) and each piece's (m, l);
//   weights_finish_kernel  joins a sequence's (m, l), reads the scores, adds the rows' weights
//                          in their order and writes decay * prior + sum.
// A key's bytes bound it: what decode reads without the values.  16 x <= 8192 tokens, 32/8 heads of 128 (139 MB): 38.0 us
// for both, 29 of them the first; with the queries as the MMA's rows it was 49.4.
//
// more rows (a window of a prompt): weights_tc.cuh, 128 at a time.
//
// All go along a line of tiles (seg_plan.cuh) of (sequence, KV head).
#pragma once

#include "seg_kernel.cuh"

namespace da {

struct WeightsParams {
  SegParams s;  // k: bf16 or int8; base = rt_prefix = 0, rt = 1
  const float* k_scale;
  const float* prior;
  float* out;
  float* scores;  // [tile of the line][64][score_rows(rows)]
  int rows;       // query rows of a KV head, or of this window
  int row0;       // the window's first
  int finish_ctas;
  float decay;
  unsigned long long timeout_ns;
};

// Rows of a token's scores in memory: whole 16 bytes.
__host__ __device__ constexpr int score_rows(int rows) { return (rows + 3) & ~3; }

template <int D, bool INT8, int NT>
struct ScoreGeo {
  static constexpr int WARPS = 4, THREADS = 32 * WARPS;
  static constexpr int ROWS = 8 * NT;           // query rows of a unit
  static constexpr int ROWB = D * (INT8 ? 1 : 2);
  static constexpr int STAGE = 16 * ROWB + (INT8 ? 64 : 0);  // keys of 16 tokens, and their scales
  // 150 KB and more of keys in flight an SM, by as many warps as their registers allow
  static constexpr int PER_SM = D == 256 ? 2 : 4;
  static constexpr int NSTAGE = ROWB == 512 ? 3 : ROWB == 256 ? (PER_SM == 2 ? 6 : 3) : 6;
  static constexpr int WARP_BYTES = NSTAGE * STAGE;
  static constexpr int OFF_ML = WARPS * WARP_BYTES;
  static constexpr int OFF_LENS = OFF_ML + WARPS * ROWS * 8;
  static constexpr int SMEM = OFF_LENS + kSegLens * 4;
};

// Where a token's row lies: its page (or sequence) and place in it.
struct Cell {
  long long slab;
  int at;
  bool good;  // a page of the pool
};
template <bool PAGED>
__device__ __forceinline__ Cell token_cell(const int* table, int max_pages, int page_size, int num_pages, int b, int t) {
  if constexpr (PAGED) {
    // (a shift where it can be one: a division is a score of instructions)
    const int col = (page_size & (page_size - 1)) == 0 ? t >> (31 - __clz(page_size)) : (int)((unsigned)t / (unsigned)page_size);
    const int page = load_dependent(table + (size_t)b * max_pages + col);
    const bool good = (unsigned)page < (unsigned)num_pages;
    if (!good) atomicOr(&g_error_word, 4u);
    return {good ? page : 0, t - col * page_size, good};
  } else {
    return {b, t, true};
  }
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Two bytes of w (from bit 16 HI) as bf16x2, exactly: 0x4300 + the low 7 bits is 128 + them,
// less 128 or, for a negative byte (whose low 7 bits are 128 + it), 256.
template <int HI>
__device__ __forceinline__ uint32_t int8x2_to_bf16x2(uint32_t w) {
  const uint32_t u = __byte_perm(w, 0u, HI ? 0x4342 : 0x4140);  // one byte a half
  const uint32_t a = (u & 0x007f007fu) | 0x43004300u, s = (u & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 d =
      __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&s));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// A warp's ring of keys: 16 tokens of every tile of the CTA's, looked up a tile ahead.
template <int D, bool PAGED, bool INT8, int NT>
struct KeyRing {
  using Gm = ScoreGeo<D, INT8, NT>;
  static constexpr int CH = Gm::ROWB / 16;  // chunks a row
  const WeightsParams& wp;
  const SegWalk<kSegRange>& walk;
  uint32_t at;  // of the ring in shared memory
  SegUnit u;
  int j;
  long long x, x1;
  // which of the 16 tokens there are, of the last eight tiles: tile x in bits 16 (x % 4) on
  unsigned long long lives0, lives1;
  int slab, row, h;  // the first one's page (not checked yet) or sequence, place in it, and head
  uint32_t live;

  __device__ __forceinline__ KeyRing(const WeightsParams& wp_, const SegWalk<kSegRange>& walk_, uint32_t at_, long long x0,
                                     long long x1_)
      : wp(wp_), walk(walk_), at(at_), x(x0), x1(x1_), lives0(0ull), lives1(0ull) {
    u = walk.at(x0, j);
    look_up();
  }
  __device__ __forceinline__ uint32_t live_of(long long tile) const {
    const int k = (int)(tile & 7);
    return (uint32_t)((k < 4 ? lives0 : lives1) >> (16 * (k & 3))) & 0xffffu;
  }
  // int8: rows 2 p and 2 p + 1 of a quarter warp's read in different halves of 128 bytes
  static __device__ __forceinline__ int chunk(int row, int c) {
    return INT8 ? c ^ ((row & 1) << 2) % CH : c ^ (row & 7);
  }
  // Starts the load of the page (16 tokens from a multiple of 16 on lie in one), which issue() uses a tile later.
  __device__ __forceinline__ void look_up() {
    const SegParams& p = wp.s;
    const int t = j * kTile + (threadIdx.x >> 5) * 16, n = u.end - t;
    live = n <= 0 ? 0u : n < 16 ? (1u << n) - 1u : 0xffffu;
    h = u.h;
    slab = u.b;
    row = t;
    if (PAGED && live) {
      const int col = t / p.page_size;
      row = t - col * p.page_size;
      slab = load_dependent(p.page_table + (size_t)u.b * p.max_pages + col);
    }
  }
  __device__ __forceinline__ void issue(int stage) {
    if (x < x1) {
      const int lane = threadIdx.x & 31, k = (int)(x & 7), bit = 16 * (k & 3);
      const unsigned long long others = ~(0xffffull << bit), mine = (unsigned long long)live << bit;
      if (k < 4)
        lives0 = (lives0 & others) | mine;
      else
        lives1 = (lives1 & others) | mine;
      if (live) {
        if (PAGED && (unsigned)slab >= (unsigned)wp.s.num_pages) {
          atomicOr(&g_error_word, 4u);
          slab = 0;
        }
        const int slab_rows = PAGED ? wp.s.page_size : wp.s.ctx;
        const long long off = (((long long)slab * slab_rows + row) * wp.s.Hkv + h) * Gm::ROWB,
                        soff = ((long long)slab * wp.s.Hkv + h) * slab_rows + row;
        const uint8_t* keys = reinterpret_cast<const uint8_t*>(wp.s.k);
        constexpr int RPP = 32 / (CH < 32 ? CH : 32);
        const int c = lane % CH, r0 = lane / CH, step = wp.s.Hkv * Gm::ROWB;
        const uint8_t* src = keys + off + r0 * step + c * 16;
        const uint32_t dst = at + stage * Gm::STAGE + r0 * Gm::ROWB;
        if (live == 0xffffu) {
#pragma unroll
          for (int r = 0; r < 16; r += RPP) {
            cp_async16(dst + r * Gm::ROWB + (chunk(r + r0, c) << 4), src, true);
            src += RPP * step;
          }
        } else {
#pragma unroll 1
          for (int r = 0; r < 16; r += RPP) {
            const bool is = (live >> (r + r0)) & 1;
            cp_async16(dst + r * Gm::ROWB + (chunk(r + r0, c) << 4), is ? src : keys, is);
            src += RPP * step;
          }
        }
        if (INT8 && lane < 16 && (live >> lane) & 1)
          cp_async4(at + stage * Gm::STAGE + 16 * Gm::ROWB + lane * 4, wp.k_scale + soff + lane);
      }
      ++x;
      if (x < x1) {
        if (++j == u.tiles) {
          u = walk.next(u);
          j = 0;
        }
        look_up();
      }
    }
    cp_async_commit();
  }
  // Step kk's fragment of a stage's 16 tokens: 0 .. 7 and 8 .. 15 in its first half of the elements, then
  // in its second.  bf16: element 16 kk + 2 t (and + 8) is thread t's of the quad; int8: 64 c + 16 t + 4 s
  // (and + 2) for kk = 4 c + s, so that a thread's 16 bytes of a key hold its elements of 4 steps, [c][row half].
  static constexpr int kHeld = INT8 ? D / 64 : 1;
  __device__ __forceinline__ void hold(int stage, uint32_t (&e)[kHeld][2][4]) const {
    if constexpr (INT8) {
      const int lane = threadIdx.x & 31;
      const uint32_t kst = at + stage * Gm::STAGE;
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int row = hf * 8 + lane / 4;
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(e[c][hf][0]), "=r"(e[c][hf][1]), "=r"(e[c][hf][2]), "=r"(e[c][hf][3])
                       : "r"(kst + row * Gm::ROWB + chunk(row, 4 * c + lane % 4) * 16));
        }
    }
  }
  __device__ __forceinline__ void fragment(int stage, int kk, const uint32_t (&e)[kHeld][2][4], uint32_t (&a)[4]) const {
    if constexpr (INT8) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        a[hf] = int8x2_to_bf16x2<0>(e[kk / 4][hf][kk % 4]);
        a[2 + hf] = int8x2_to_bf16x2<1>(e[kk / 4][hf][kk % 4]);
      }
    } else {
      const int lane = threadIdx.x & 31, row = lane & 15, c = 2 * kk + (lane >> 4);
      ldsm_x4(at + stage * Gm::STAGE + row * Gm::ROWB + (chunk(row, c) << 4), a[0], a[1], a[2], a[3]);
    }
  }
  // The words of a query row (32-bit index) that go with them for step kk: first and second half.
  static __device__ __forceinline__ int query_word(int kk, int t) {
    return INT8 ? 32 * (kk / 4) + 8 * t + 2 * (kk % 4) : 8 * kk + t;
  }
  static constexpr int kQueryHalf = INT8 ? 1 : 4;
};

// Joins the warps' (m, l) of a row.
template <int WARPS, int ROWS>
__device__ __forceinline__ float2 join_warps(const float2* ml, int row) {
  float M = kNegInf, L = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) M = fmaxf(M, ml[w * ROWS + row].x);
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const float2 y = ml[w * ROWS + row];
    if (y.y != 0.f) L += y.x == kNegInf ? y.y : exp2_approx(y.x - M) * y.y;
  }
  return make_float2(M, L);
}

// The tokens are the MMA's 16 rows and the queries its 8 columns, as in seg_kernel.  A lane keeps a
// maximum and a sum of its own tokens; the lanes are joined where a unit ends.
template <int D, bool PAGED, bool INT8, int NT>
__global__ void __launch_bounds__(ScoreGeo<D, INT8, NT>::THREADS, ScoreGeo<D, INT8, NT>::PER_SM)
    weights_score_kernel(const __grid_constant__ WeightsParams wp) {
  using Gm = ScoreGeo<D, INT8, NT>;
  using Ring = KeyRing<D, PAGED, INT8, NT>;
  const SegParams& p = wp.s;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_wait_primary();
  pdl_launch_dependents();
  const SegWalk<kSegRange> walk(p, seg_stage_lens<Gm::THREADS>(p, reinterpret_cast<int*>(smem + Gm::OFF_LENS)));
  long long x0, x1;
  if (!walk.range(blockIdx.x, x0, x1)) return;
  Ring ring(wp, walk, smem_u32(smem + warp * Gm::WARP_BYTES), x0, x1);
  SegUnit u = ring.u;
  int j = ring.j;
#pragma unroll 1
  for (int s = 0; s < Gm::NSTAGE; ++s) ring.issue(s);

  // column n of an MMA is row 8 nt + n; this lane's columns are 2 (lane % 4) and the next
  uint32_t qb[NT][D / 16][2];
  float m[NT][2], l[NT][2];
  int lim[NT][2];
  const int padded = score_rows(wp.rows);
  bool fresh = true;
  int stage = 0;
  for (long long x = x0; x < x1; ++x) {
    if (fresh) {
      fresh = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        int token, g, unused;
        const bool is = seg_query<kSegRange>(p, walk.lens, u, 8 * nt + lane / 4, token, g, unused);
        const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + ((size_t)token * p.Hq + u.h * p.G + g) * D);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int w = Ring::query_word(kk, lane % 4);
          qb[nt][kk][0] = is ? load_dependent(src + w) : 0u;
          qb[nt][kk][1] = is ? load_dependent(src + w + Ring::kQueryHalf) : 0u;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          seg_query<kSegRange>(p, walk.lens, u, 8 * nt + 2 * (lane % 4) + e, token, g, lim[nt][e]);  // 0: no row
          m[nt][e] = kNegInf;
          l[nt][e] = 0.f;
        }
      }
    }
    cp_async_wait<Gm::NSTAGE - 1>();
    __syncwarp();
    const uint32_t live = ring.live_of(x);
    if (live) {
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
      uint32_t held[Ring::kHeld][2][4];
      ring.hold(stage, held);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t a[4];
        ring.fragment(stage, kk, held, a);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(s[nt], a[0], a[1], a[2], a[3], qb[nt][kk][0], qb[nt][kk][1]);
      }
      float* to = wp.scores + ((size_t)x * kTile + warp * 16 + lane / 4) * padded + 2 * (lane % 4);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float f = p.scale_log2;
        if (INT8) f *= *reinterpret_cast<const float*>(smem + warp * Gm::WARP_BYTES + stage * Gm::STAGE + 16 * Gm::ROWB +
                                                       (lane / 4 + 8 * hf) * 4);
        const int t = j * kTile + warp * 16 + lane / 4 + 8 * hf;
        const bool is = (live >> (lane / 4 + 8 * hf)) & 1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) s[nt][2 * hf + e] = is && t < lim[nt][e] ? s[nt][2 * hf + e] * f : kNegInf;
          if (8 * nt + 2 * (lane % 4) < padded)
            *reinterpret_cast<float2*>(to + 8 * hf * padded + 8 * nt) = make_float2(s[nt][2 * hf], s[nt][2 * hf + 1]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mx = fmaxf(s[nt][e], s[nt][2 + e]);
          if (mx > m[nt][e]) {
            l[nt][e] *= exp2_approx(m[nt][e] - mx);
            m[nt][e] = mx;
          }
          const float mu = m[nt][e] == kNegInf ? 0.f : m[nt][e];
          l[nt][e] += exp2_approx(s[nt][e] - mu) + exp2_approx(s[nt][2 + e] - mu);
        }
    }
    const bool last = j + 1 == u.tiles;
    if (last || x + 1 == x1) {
      float2* ml = reinterpret_cast<float2*>(smem + Gm::OFF_ML);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = m[nt][e];
#pragma unroll
          for (int d = 4; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          float sum = m[nt][e] == kNegInf ? l[nt][e] : l[nt][e] * exp2_approx(m[nt][e] - top);  // 0, or NaN
#pragma unroll
          for (int d = 4; d < 32; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          if (lane < 4) ml[warp * Gm::ROWS + 8 * nt + 2 * lane + e] = make_float2(top, sum);
        }
      __syncthreads();
      if (threadIdx.x < Gm::ROWS)
        p.part_ml[((size_t)u.id + blockIdx.x) * 16 + threadIdx.x] = join_warps<Gm::WARPS, Gm::ROWS>(ml, threadIdx.x);
      __syncthreads();
    }
    __syncwarp();  // every lane has read its tokens' scales: their place is filled again
    ring.issue(stage);
    stage = stage + 1 == Gm::NSTAGE ? 0 : stage + 1;
    ++j;
    if (last && x + 1 < x1) {
      u = walk.next(u);
      j = 0;
      fresh = true;
    }
  }
  cp_async_wait<0>();
}

// (m, l) of row r of a unit from its pieces, [slot][stride] of them; the warp executes it.
__device__ __forceinline__ float2 join_pieces(const float2* ml, long long slot, int pieces, int stride, int r) {
  const int lane = threadIdx.x & 31;
  float M = kNegInf, L = 0.f;
  for (int k = lane; k < pieces; k += 32) {
    const float2 y = __ldcg(ml + (slot + k) * stride + r);
    if (y.y == 0.f) continue;
    const float to = fmaxf(M, y.x);
    L = (M == kNegInf ? L : L * exp2_approx(M - to)) + (y.x == kNegInf ? y.y : y.y * exp2_approx(y.x - to));
    M = to;
  }
  float top = M;
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  L = M == kNegInf ? L : L * exp2_approx(M - top);
#pragma unroll
  for (int d = 16; d; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
  return make_float2(top, L);
}
// What a weight is made with: 2^(x - .x) * .y; a row that saw nothing gives nothing.
__device__ __forceinline__ float2 weight_factors(float2 ml) {
  return make_float2(ml.x == kNegInf ? 0.f : ml.x, ml.y == 0.f ? 0.f : 1.f / ml.y);
}

// A thread a token: it adds the rows in their order, 256 tokens of a sequence's KV head at a time.
// The plan, the pages and the priors come before the wait: nothing that weights_score_kernel
// writes is among them, and the kernels before that one were done when it let this one start.
constexpr int kFinishThreads = 256;

template <bool PAGED>
__global__ void __launch_bounds__(kFinishThreads) weights_finish_kernel(const __grid_constant__ WeightsParams wp) {
  const SegParams& p = wp.s;
  __shared__ float2 row[16];
  __shared__ int s_lens[kSegLens];
  const int* lens = seg_stage_lens<kFinishThreads>(p, s_lens);
  const long long all = seg_sums(lens, p.B, p.cap, 0, 0).all;  // tiles of the batch
  const long long W = all * p.Hkv;
  const int used = seg_used(W, p.ctas), ctas = seg_used(W, wp.finish_ctas);
  long long f = 0, f1 = 0;
  if ((int)blockIdx.x < ctas) {
    f = seg_start(W, ctas, blockIdx.x);
    f1 = seg_start(W, ctas, blockIdx.x + 1);
  }
  bool waited = false;
  while (f < f1) {
    const SegAt s = seg_find(lens, p.B, p.cap, 0, seg_div(f, p.Hkv));
    const int L = seg_len(lens, s.b, p.cap), tiles = seg_tiles(L, p.cap, 0);
    const int h = (int)seg_div(f - s.start * p.Hkv, tiles), j0 = (int)(f - s.start * p.Hkv - (long long)h * tiles);
    const int j1 = (int)min((long long)tiles, j0 + (f1 - f));
    const long long line = s.start * p.Hkv + (long long)h * tiles;  // its first tile among the scores
    const int c0 = seg_owner(W, used, line), c1 = seg_owner(W, used, line + tiles - 1);
    bool fresh = true;
    for (int ja = j0; ja < j1; ja += kFinishThreads / kTile) {
      const int j = ja + threadIdx.x / kTile, t = j * kTile + threadIdx.x % kTile;
      const bool mine = j < j1 && t < L;
      Cell c = {0, 0, false};
      size_t o = 0;
      float before = 0.f;
      if (mine) {
        c = token_cell<PAGED>(p.page_table, p.max_pages, p.page_size, p.num_pages, s.b, t);
        o = ((size_t)c.slab * p.Hkv + h) * (PAGED ? p.page_size : p.ctx) + c.at;
        if (wp.prior && c.good) before = load_dependent(wp.prior + o);
      }
      if (!waited) {
        waited = true;
        pdl_wait_primary();
      }
      if (fresh) {
        fresh = false;
        __syncthreads();
        for (int r = threadIdx.x >> 5; r < 16; r += kFinishThreads / 32) {
          float2 y = make_float2(0.f, 0.f);
          if (r < wp.rows) y = weight_factors(join_pieces(p.part_ml, (long long)(s.b * p.Hkv + h) + c0, c1 - c0 + 1, 16, r));
          if ((threadIdx.x & 31) == 0) row[r] = y;
        }
        __syncthreads();
      }
      if (!mine) continue;
      const float4* x = reinterpret_cast<const float4*>(wp.scores + ((size_t)(line + j) * kTile + threadIdx.x % kTile) *
                                                                        score_rows(wp.rows));
      // The rows that see the token are those from `from` on (rows past the last: score -inf, factor 0); the others' scores are
      // -inf, but a row's factor may be NaN.
      const int from = max(t - (L - p.n), 0) * p.G;
      float w = 0.f;
#pragma unroll 2
      for (int r = from & ~3; r < wp.rows; r += 4) {
        const float4 y = __ldcg(x + r / 4);
        w = fmaf(exp2_approx(y.x - row[r].x), r >= from ? row[r].y : 0.f, w);
        w = fmaf(exp2_approx(y.y - row[r + 1].x), r + 1 >= from ? row[r + 1].y : 0.f, w);
        w = fmaf(exp2_approx(y.z - row[r + 2].x), r + 2 >= from ? row[r + 2].y : 0.f, w);
        w = fmaf(exp2_approx(y.w - row[r + 3].x), row[r + 3].y, w);  // (from is less than r + 4)
      }
      if (c.good) wp.out[o] = wp.prior ? fmaf(wp.decay, before, w) : w;
    }
    f += j1 - j0;
  }
  if (!waited) pdl_wait_primary();
}

}  // namespace da
