// The attention weight that new tokens give each cached token, summed over them and over the
// heads of a group.  A softmax needs its whole row's maximum and sum before the first weight
// is known, so there are two kernels:
//   scores    reads every key once, 16 query rows at a time on the warp-level MMA, writes the
//             scores (64 fp32 a row and tile, a sixteenth of a bf16 key's bytes a row) and
//             each piece's (m, l);
//   finish    joins a sequence's (m, l), reads the scores, adds the rows' weights in their
//             order and writes decay * prior + sum.
// Both go along a line of tiles (seg_plan.cuh), of (sequence, KV head, 16 rows) and of (sequence,
// KV head).  A key's bytes bound it: what decode reads without the values.
#pragma once

#include "seg_kernel.cuh"

namespace da {

struct WeightsParams {
  SegParams s;  // k: bf16 or int8; base = rt_prefix = 0
  const float* k_scale;
  const float* prior;
  float* out;
  float* scores;  // [tile of the line][rows of a unit, 16 at most][64]
  int rows;       // that number
  int finish_ctas;
  float decay;
};

template <int D, bool INT8>
struct ScoreGeo {
  static constexpr int WARPS = 4, THREADS = 32 * WARPS;
  static constexpr int ROWB = D * (INT8 ? 1 : 2);
  static constexpr int STAGE = 16 * ROWB + (INT8 ? 64 : 0);  // keys of 16 tokens, and their scales
  static constexpr int NSTAGE = ROWB == 512 ? 3 : 6;  // two CTAs an SM either way
  static constexpr int WARP_BYTES = NSTAGE * STAGE;
  static constexpr int OFF_ML = WARPS * WARP_BYTES;
  static constexpr int OFF_MASK = OFF_ML + WARPS * 16 * 8;
  static constexpr int OFF_LENS = OFF_MASK + WARPS * NSTAGE * 4;
  static constexpr int SMEM = OFF_LENS + kSegLens * 4;
  static constexpr int PER_SM = 2;
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
    const int col = t / page_size;
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

template <int D, bool PAGED, bool INT8>
__global__ void __launch_bounds__(ScoreGeo<D, INT8>::THREADS, ScoreGeo<D, INT8>::PER_SM)
    weights_score_kernel(const __grid_constant__ WeightsParams wp) {
  using Gm = ScoreGeo<D, INT8>;
  const SegParams& p = wp.s;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * Gm::WARP_BYTES;
  const uint32_t ring_s = smem_u32(ring);
  volatile uint32_t* masks = reinterpret_cast<volatile uint32_t*>(smem + Gm::OFF_MASK) + warp * Gm::NSTAGE;

  pdl_wait_primary();
  pdl_launch_dependents();
  const SegWalk<kSegRange> walk(p, seg_stage_lens<Gm::THREADS>(p, reinterpret_cast<int*>(smem + Gm::OFF_LENS)));
  long long x0, x1;
  if (!walk.range(blockIdx.x, x0, x1)) return;

  const uint8_t* keys = reinterpret_cast<const uint8_t*>(p.k);
  const int slab_rows = PAGED ? p.page_size : p.ctx;
  int lj;
  SegUnit lu = walk.at(x0, lj);
  long long lx = x0, off = -1, soff = 0;
  auto look_up = [&]() {
    off = -1;
    const int t = lj * kTile + warp * 16 + lane;
    if (lane < 16 && t < lu.end) {
      const Cell c = token_cell<PAGED>(p.page_table, p.max_pages, p.page_size, p.num_pages, lu.b, t);
      off = ((c.slab * slab_rows + c.at) * p.Hkv + lu.h) * (long long)Gm::ROWB;
      soff = (c.slab * p.Hkv + lu.h) * slab_rows + c.at;
    }
  };
  look_up();
  auto issue = [&](int stage) {
    if (lx < x1) {
      const uint32_t live = __ballot_sync(0xffffffffu, off >= 0);
      if (lane == 0) masks[stage] = live;
      if (live) {
        const uint32_t dst = ring_s + stage * Gm::STAGE;
        constexpr int CH = Gm::ROWB / 16, RPP = 32 / (CH < 32 ? CH : 32);
        const int c = lane % CH, r0 = lane / CH;
#pragma unroll
        for (int r = 0; r < 16; r += RPP) {
          const int row = r + r0;
          const long long o = __shfl_sync(0xffffffffu, off, row);
          // int8: rows 2 p and 2 p + 1 of a quarter warp's read in different halves of 128 bytes
          const int at = INT8 ? c ^ ((row & 1) << 2) % CH : c ^ (row & 7);
          cp_async16(dst + row * Gm::ROWB + (at << 4), keys + (o < 0 ? 0 : o) + c * 16, o >= 0);
        }
        if (INT8 && off >= 0) cp_async4(dst + 16 * Gm::ROWB + lane * 4, wp.k_scale + soff);
      }
      ++lx;
      if (lx < x1) {
        if (++lj == lu.tiles) {
          lu = walk.next(lu);
          lj = 0;
        }
        look_up();
      }
    }
    cp_async_commit();
  };

  int j = lj;
  SegUnit u = lu;
#pragma unroll 1
  for (int s = 0; s < Gm::NSTAGE; ++s) issue(s);

  uint32_t qa[D / 16][4];
  float m[2], l[2];
  int lim[2];
  bool has[2];
  bool fresh = true;
  int stage = 0;
  for (long long x = x0; x < x1; ++x) {
    if (fresh) {
      fresh = false;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        int token, g;
        has[hf] = seg_query<kSegRange>(p, walk.lens, u, lane / 4 + 8 * hf, token, g, lim[hf]);
        const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + ((size_t)token * p.Hq + u.h * p.G + g) * D);
        // bf16: element 16 kk + 2 t (and + 8) is thread t's of the quad; int8: 64 c + 16 t + 4 s (and
        // + 2) for kk = 4 c + s, so that a thread's 16 bytes of a key hold its elements of 4 steps
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int w = INT8 ? 32 * (kk / 4) + 8 * (lane % 4) + 2 * (kk % 4) : 8 * kk + lane % 4;
          qa[kk][hf] = has[hf] ? load_dependent(src + w) : 0u;
          qa[kk][2 + hf] = has[hf] ? load_dependent(src + w + (INT8 ? 1 : 4)) : 0u;
        }
        m[hf] = kNegInf;
        l[hf] = 0.f;
      }
    }
    cp_async_wait<Gm::NSTAGE - 1>();
    __syncwarp();
    const uint32_t live = masks[stage];
    if (live) {
      const uint32_t kst = ring_s + stage * Gm::STAGE;
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      float ks[2][2] = {{1.f, 1.f}, {1.f, 1.f}};
      if constexpr (INT8) {
        constexpr int CH = Gm::ROWB / 16;
        const uint8_t* kp = ring + stage * Gm::STAGE;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int row = nt * 8 + lane / 4;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const int ch = (4 * c + lane % 4) ^ ((row & 1) << 2) % CH;
            const uint4 w = *reinterpret_cast<const uint4*>(kp + row * Gm::ROWB + ch * 16);
            const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_bf16_16816(s[nt], qa[4 * c + i][0], qa[4 * c + i][1], qa[4 * c + i][2], qa[4 * c + i][3],
                             int8x2_to_bf16x2<0>(e[i]), int8x2_to_bf16x2<1>(e[i]));
          }
          const float2 sc = *reinterpret_cast<const float2*>(kp + 16 * Gm::ROWB + (nt * 8 + 2 * (lane % 4)) * 4);
          ks[nt][0] = sc.x;
          ks[nt][1] = sc.y;
        }
      } else {
        const int mrow = lane & 7, mi = lane >> 3;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t r0, r1, r2, r3;
          const int row = (mi >> 1) * 8 + mrow, c = 2 * kk + (mi & 1);
          ldsm_x4(kst + row * Gm::ROWB + ((c ^ mrow) << 4), r0, r1, r2, r3);
          mma_bf16_16816(s[0], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], r0, r1);
          mma_bf16_16816(s[1], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], r2, r3);
        }
      }
      float mx[2] = {kNegInf, kNegInf};
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = nt * 8 + 2 * (lane % 4) + (e & 1);
          const bool see = ((live >> col) & 1) && j * kTile + warp * 16 + col < lim[e >> 1];
          s[nt][e] = see ? s[nt][e] * ks[nt][e & 1] * p.scale_log2 : kNegInf;
          mx[e >> 1] = fmaxf(mx[e >> 1], s[nt][e]);
        }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 1));
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 2));
        if (mx[hf] > m[hf]) {
          l[hf] *= exp2_approx(m[hf] - mx[hf]);
          m[hf] = mx[hf];
        }
        const float mu = m[hf] == kNegInf ? 0.f : m[hf];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          l[hf] += exp2_approx(s[nt][2 * hf] - mu) + exp2_approx(s[nt][2 * hf + 1] - mu);
          if (has[hf])
            *reinterpret_cast<float2*>(wp.scores + ((size_t)x * wp.rows + lane / 4 + 8 * hf) * kTile + warp * 16 + nt * 8 +
                                       2 * (lane % 4)) = make_float2(s[nt][2 * hf], s[nt][2 * hf + 1]);
        }
      }
    }
    const bool last = j + 1 == u.tiles;
    if (last || x + 1 == x1) {
      float2* ml = reinterpret_cast<float2*>(smem + Gm::OFF_ML);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 1);
        l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 2);
        if (lane % 4 == 0) ml[warp * 16 + lane / 4 + 8 * hf] = make_float2(m[hf], l[hf]);
      }
      __syncthreads();
      if (threadIdx.x < 16) {
        float M = kNegInf, L = 0.f;
#pragma unroll
        for (int w = 0; w < Gm::WARPS; ++w) M = fmaxf(M, ml[w * 16 + threadIdx.x].x);
#pragma unroll
        for (int w = 0; w < Gm::WARPS; ++w) {
          const float2 y = ml[w * 16 + threadIdx.x];
          if (y.y != 0.f) L += y.x == kNegInf ? y.y : exp2_approx(y.x - M) * y.y;
        }
        p.part_ml[((size_t)u.id + blockIdx.x) * 16 + threadIdx.x] = make_float2(M, L);
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
}

constexpr int kFinishThreads = 256, kFinishRows = 1024;

template <bool PAGED>
__global__ void __launch_bounds__(kFinishThreads) weights_finish_kernel(const __grid_constant__ WeightsParams wp) {
  const SegParams& p = wp.s;
  __shared__ float2 row_ml[kFinishRows];  // m and 1 / l
  __shared__ float sums[kFinishThreads];
  pdl_wait_primary();
  const long long all = seg_sums(p.seq_lens, p.B, p.cap, 0, 0).all;  // tiles of the batch
  const long long W = all * p.Hkv * p.rt, F = all * p.Hkv;
  const long long f0 = seg_start(F, wp.finish_ctas, blockIdx.x), f1 = seg_start(F, wp.finish_ctas, blockIdx.x + 1);
  const int rows = p.n * p.G, used = seg_used(W, p.ctas);
  long long f = f0;
  while (f < f1) {  // a sequence's KV head at a time
    const SegAt s = seg_find(p.seq_lens, p.B, p.cap, 0, f / p.Hkv);
    const int L = seg_len(p.seq_lens, s.b, p.cap), tiles = seg_tiles(L, p.cap, 0);
    const int h = (int)((f - s.start * p.Hkv) / tiles), j0 = (int)((f - s.start * p.Hkv) % tiles);
    const int j1 = (int)min((long long)tiles, j0 + (f1 - f));
    const long long line = s.start * p.Hkv * p.rt + (long long)h * p.rt * tiles;  // its first tile among the scores
    __syncthreads();
    for (int r = threadIdx.x; r < rows; r += kFinishThreads) {
      const long long a = line + (long long)(r / 16) * tiles;
      const int c0 = seg_owner(W, used, a), c1 = seg_owner(W, used, a + tiles - 1);
      const float2* ml = p.part_ml + ((size_t)(s.b * p.Hkv + h) * p.rt + r / 16 + c0) * 16 + r % 16;
      float M = kNegInf, sum = 0.f;
#pragma unroll 4
      for (int k = 0; k <= c1 - c0; ++k) {
        const float2 y = __ldcg(ml + (size_t)k * 16);
        if (y.y == 0.f) continue;
        const float to = fmaxf(M, y.x);
        sum = (M == kNegInf ? sum : sum * exp2_approx(M - to)) + (y.x == kNegInf ? y.y : y.y * exp2_approx(y.x - to));
        M = to;
      }
      row_ml[r] = make_float2(M == kNegInf ? 0.f : M, sum == 0.f ? 0.f : 1.f / sum);
    }
    __syncthreads();
    const int at = threadIdx.x % kTile, part = threadIdx.x / kTile;
    constexpr int PARTS = kFinishThreads / kTile;
    for (int j = j0; j < j1; ++j) {
      const int t = j * kTile + at;
      float w = 0.f;
      if (t < L) {
#pragma unroll 4
        for (int r = part; r < rows; r += PARTS) {
          const float x = __ldcg(wp.scores + ((size_t)(line + (long long)(r / 16) * tiles + j) * wp.rows + r % 16) * kTile + at);
          w += exp2_approx(x - row_ml[r].x) * row_ml[r].y;
        }
      }
      sums[threadIdx.x] = w;
      __syncthreads();
      if (part == 0 && t < L) {
#pragma unroll
        for (int k = 1; k < PARTS; ++k) w += sums[k * kTile + at];
        const Cell c = token_cell<PAGED>(p.page_table, p.max_pages, p.page_size, p.num_pages, s.b, t);
        if (c.good) {
          const size_t o = ((size_t)c.slab * p.Hkv + h) * (PAGED ? p.page_size : p.ctx) + c.at;
          wp.out[o] = wp.prior ? fmaf(wp.decay, load_dependent(wp.prior + o), w) : w;
        }
      }
      __syncthreads();
    }
    f += j1 - j0;
  }
}

}  // namespace da
