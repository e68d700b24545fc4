// The attention weights of a window of many query rows on the 5th-generation tensor cores.
//
// 128 query rows of a KV head at a time (q_len tokens x G heads), against all of its keys, twice:
//   !SUMS  S = Q K^T, a row a lane of tensor memory: its maximum and sum over this CTA's keys;
//   SUMS   S^T = K Q^T, a token a lane: w_t = sum_r 2^(s_rt - m_r) / l_r, with (m, l) of all CTAs.
// The scores are computed twice: writing and reading 128 fp32 a key costs more than its 128 to 512
// bytes.  2 x 2 D operations a (row, key) on tcgen05 and two exponentials: 32 tokens x 32 heads over
// 32768 keys are 9 us of operations and 15 of exponentials (warp-level MMAs, at 256 products a
// cycle and SM, take 58 us a pass); measured, 49.4 for both.  Latency bounds them: a CTA has about seven tiles a pass, 3.7 us each,
// with one tile's loads in flight.  Both operands lie K-major in shared memory, so that the two passes differ in which is A.
//
// Warps 0 to 3 bring the keys: they look a tile's tokens up, load them, widen int8, and store
// them with the swizzle of the products, two tiles of 128 tokens deep; warp 8 issues the products
// into two buffers of tensor memory; warps 4 to 7 take a buffer's lanes, a thread each.  Two CTAs
// an SM (one at D = 256), so that one's exponentials run beside the other's loads.
#pragma once

#include "tc05.cuh"
#include "weights_kernel.cuh"

namespace da {

template <int D>
struct WeightsTcGeo {
  static constexpr int ROWS = 128, KEYS = 128;
  static constexpr int THREADS = 288;
  static constexpr int TILE = 128 * D * 2;  // 128 rows of either operand, [D / 64][128][64]
  static constexpr int OFF_K = TILE, OFF_OFF = OFF_K + 2 * TILE;  // queries, then two tiles of keys
  static constexpr int OFF_KS = OFF_OFF + 2 * KEYS * 8;           // where their tokens lie; scales of eight tiles
  static constexpr int OFF_F = OFF_KS + 8 * KEYS * 4;             // factors of the rows
  static constexpr int BAR_KF = 0, BAR_KE = 2, BAR_SF = 4, BAR_SE = 6, BAR_FIN = 8;
  static constexpr int OFF_BAR = OFF_F + ROWS * 8;
  static constexpr int OFF_MISC = OFF_BAR + 9 * 8 + 8;  // tensor memory base, abort flag
  static constexpr int OFF_LENS = OFF_MISC + 16;
  static constexpr int SMEM = OFF_LENS + kSegLens * 4 + 1024;
  static constexpr int PER_SM = D == 256 ? 1 : 2;
};

template <int D, bool PAGED, bool INT8, bool SUMS>
__global__ void __launch_bounds__(WeightsTcGeo<D>::THREADS, WeightsTcGeo<D>::PER_SM)
    weights_tc_kernel(const __grid_constant__ WeightsParams wp) {
  using Gm = WeightsTcGeo<D>;
  const SegParams& p = wp.s;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  auto bar = [&](int i) -> uint32_t { return sbase + Gm::OFF_BAR + 8 * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Gm::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(Gm::BAR_KF + i), 128);
      mbar_init(bar(Gm::BAR_KE + i), 1);
      mbar_init(bar(Gm::BAR_SF + i), 2);  // the products, and who issued them (for the scales)
      mbar_init(bar(Gm::BAR_SE + i), 128);
    }
    mbar_init(bar(Gm::BAR_FIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // Tensor memory is taken after the wait and before the next kernel may start: none waits for another
  // while it holds some that the other still has to take.
  pdl_wait_primary();
  if (warp == 8) {
    tmem_alloc(sbase + Gm::OFF_MISC, 256);
    tmem_relinquish();
  }
  const SegWalk<kSegRange> walk(p, seg_stage_lens<Gm::THREADS>(p, reinterpret_cast<int*>(smem + Gm::OFF_LENS)));
  long long x0 = 0, x1 = 0;
  if (!walk.range(blockIdx.x, x0, x1)) x0 = x1 = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Gm::OFF_MISC);
  auto wait = [&](int i, int phase) { return wait_bounded(bar(i), (uint32_t)(phase & 1), abort_flag, wp.timeout_ns); };

  SegUnit u = {};
  int j = 0;
  if (x0 < x1) u = walk.at(x0, j);
  int it = 0;  // tiles of 128 tokens so far
  bool ok = true, issued = false;
  for (long long x = x0; x < x1 && ok;) {
    // this CTA's tokens of the unit: [t0, t1)
    const int tiles64 = (int)min((long long)(u.tiles - j), x1 - x);
    const int t0 = j * kTile, t1 = min(u.end, (j + tiles64) * kTile);
    const int n = (t1 - t0 + Gm::KEYS - 1) / Gm::KEYS;
    // warps 0 to 3: a thread a token of tile k
    long long* offs = reinterpret_cast<long long*>(smem + Gm::OFF_OFF);
    constexpr int ROWB = D * (INT8 ? 1 : 2), CH = ROWB / 16;
    long long next_off = -1;
    float next_scale = 0.f;
    auto look_up = [&](int k) {  // starts the loads; their results are stored later
      next_off = -1;
      next_scale = 0.f;
      const int t = t0 + k * Gm::KEYS + threadIdx.x;
      if (t < t1) {
        const Cell c = token_cell<PAGED>(p.page_table, p.max_pages, p.page_size, p.num_pages, u.b, t);
        const int slab_rows = PAGED ? p.page_size : p.ctx;
        next_off = ((c.slab * slab_rows + c.at) * p.Hkv + u.h) * (long long)ROWB;
        next_scale = 1.f;
        if (INT8) next_scale = load_dependent(wp.k_scale + (c.slab * p.Hkv + u.h) * slab_rows + c.at);
      }
    };
    // The place of a tile's scales was last read for the tile eight before, long done: the products of tile
    // at - 2, which are waited for below, began after the readers of tile at - 4.
    auto keep = [&](int k) {
      offs[((it + k) & 1) * Gm::KEYS + threadIdx.x] = next_off;
      reinterpret_cast<float*>(smem + Gm::OFF_KS)[((it + k) & 7) * Gm::KEYS + threadIdx.x] = next_scale * p.scale_log2;
    };
    // Its queries (the products of the last unit's are done: every thread has seen their results).  Rows past the last one
    // are the last one again, with its m and a factor of 0: zeros there would be NaN against an infinite key, which that
    // row may well score -inf, and a NaN of its own is in the sum anyway.
    {
      constexpr int QCH = D / 8, STEP = Gm::THREADS / QCH;  // a thread's chunk of every STEP-th row
      static_assert(Gm::THREADS % QCH == 0, "");
      const int c = threadIdx.x % QCH, more = STEP / p.G, step_g = STEP - more * p.G;
      const uint32_t column = sbase + (c / 8) * 16384;
      int in = threadIdx.x / QCH, token = (wp.row0 + in) / p.G, g = wp.row0 + in - token * p.G;
      const __nv_bfloat16* from = p.q + ((size_t)u.b * p.n * p.Hq + (size_t)u.h * p.G) * D + c * 8;
      const int last = wp.row0 + wp.rows - 1, last_token = last / p.G;
      const __nv_bfloat16* again = from + ((size_t)last_token * p.Hq + (last - last_token * p.G)) * D;
#pragma unroll 4
      for (; in < Gm::ROWS; in += STEP) {
        cp_async16(column + swz<128>(in, c % 8), in < wp.rows ? from + ((size_t)token * p.Hq + g) * D : again, true);
        token += more;
        g += step_g;
        if (g >= p.G) {
          g -= p.G;
          ++token;
        }
      }
      cp_async_commit();
      if (warp < 4) {
        look_up(0);
        keep(0);
      }
      if (SUMS && warp >= 4 && warp < 8) {
        // a thread a row: its (m, l) over all pieces of the unit
        const int r = threadIdx.x - 128;
        const SegSums sums = seg_sums(walk.lens, p.B, p.cap, 0, u.b);
        const long long a = sums.before * p.Hkv + (long long)u.h * u.tiles;
        const int c0 = seg_owner(walk.all, walk.used, a), c1 = seg_owner(walk.all, walk.used, a + u.tiles - 1);
        const float2* ml = p.part_ml + ((long long)u.id + c0) * Gm::ROWS + min(r, wp.rows - 1);
        float M = kNegInf, L = 0.f;
        constexpr int U2 = 20;
        for (int k0 = 0; k0 <= c1 - c0; k0 += U2) {
          float2 y[U2];
#pragma unroll
          for (int k = 0; k < U2; ++k)
            y[k] = k0 + k <= c1 - c0 ? __ldcg(ml + (size_t)(k0 + k) * Gm::ROWS) : make_float2(kNegInf, 0.f);
          float top = M, sum = 0.f;  // (one piece after another, each with its exponentials, made a chain of 2 us)
#pragma unroll
          for (int k = 0; k < U2; ++k) top = fmaxf(top, y[k].y == 0.f ? kNegInf : y[k].x);
#pragma unroll
          for (int k = 0; k < U2; ++k)
            sum += y[k].y == 0.f ? 0.f : y[k].x == kNegInf ? y[k].y : y[k].y * exp2_approx(y[k].x - top);
          L = (M == kNegInf ? L : L * exp2_approx(M - top)) + sum;
          M = top;
        }
        float2 f = weight_factors(make_float2(M, L));
        if (r >= wp.rows) f.y = 0.f;
        float* to = reinterpret_cast<float*>(smem + Gm::OFF_F) + (r / 2) * 4 + r % 2;  // -m of two rows, then their 1 / l
        to[0] = -f.x;
        to[2] = f.y;
      }
      cp_async_wait<0>();
      fence_proxy_async_smem();
      __syncthreads();
    }

    if (warp < 4) {
      // ---- keys
      const int me = threadIdx.x;
      // (after a wait that gave up, the threads go on without waits, so that all meet at the barrier)
      for (int k = 0; k < n; ++k) {
        const int at = it + k, buf = at & 1;
        named_bar_sync(1, 128);
        const long long* off = offs + buf * Gm::KEYS;
        uint8_t* dst = smem + Gm::OFF_K + buf * Gm::TILE;
        constexpr int U = CH < 8 ? CH : Gm::PER_SM == 2 ? 8 : 16;  // loads of a thread in flight
        for (int e0 = 0; e0 < Gm::KEYS * CH; e0 += U * 128) {
          uint4 v[U];
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int row = (e0 + i * 128 + me) / CH, c = (e0 + i * 128 + me) % CH;
            const long long o = off[row];
            v[i] = o >= 0 ? load_dependent(reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(p.k) + o) + c)
                          : make_uint4(0u, 0u, 0u, 0u);
          }
          if (e0 == 0) look_up(k + 1);
          if (e0 == 0 && at >= 2) ok = ok && wait(Gm::BAR_KE + buf, (at >> 1) - 1);
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int row = (e0 + i * 128 + me) / CH, c = (e0 + i * 128 + me) % CH;
            if constexpr (INT8) {
              const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
              uint32_t y[8];
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                y[2 * z] = int8x2_to_bf16x2<0>(w[z]);
                y[2 * z + 1] = int8x2_to_bf16x2<1>(w[z]);
              }
              uint8_t* to = dst + (c / 4) * 16384;
              *reinterpret_cast<uint4*>(to + swz<128>(row, 2 * (c % 4))) = make_uint4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<uint4*>(to + swz<128>(row, 2 * (c % 4) + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
            } else {
              *reinterpret_cast<uint4*>(dst + (c / 8) * 16384 + swz<128>(row, c % 8)) = v[i];
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(Gm::BAR_KF + buf));
        keep(k + 1);
      }
    } else if (warp == 8) {
      // ---- products
      constexpr uint32_t id = tc_idesc_bf16(128, 128, false, false);
      for (int k = 0; k < n; ++k) {
        const int at = it + k, buf = at & 1;
        ok = __all_sync(0xffffffffu, wait(Gm::BAR_KF + buf, at >> 1));
        if (ok && at >= 2) ok = __all_sync(0xffffffffu, wait(Gm::BAR_SE + buf, (at >> 1) - 1));
        if (!ok) break;
        issued = true;
        if (elect_one()) {
          tc_fence_after();
          const uint32_t q = sbase, key = sbase + Gm::OFF_K + buf * Gm::TILE;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint64_t da = tc_sdesc((SUMS ? key : q) + c * 16384, 16, 1024, kTcSwizzle128B);
            const uint64_t db = tc_sdesc((SUMS ? q : key) + c * 16384, 16, 1024, kTcSwizzle128B);
#pragma unroll
            for (int i = 0; i < 4; ++i) tc_mma_ss(tmem + buf * 128, da + 2 * i, db + 2 * i, id, c > 0 || i > 0);
          }
          tc_commit(bar(Gm::BAR_KE + buf));
          tc_commit(bar(Gm::BAR_SF + buf));
          mbar_arrive(bar(Gm::BAR_SF + buf));
        }
        __syncwarp();
      }
    } else {
      // ---- exponentials: a thread a row (SUMS: a token)
      const int me = threadIdx.x - 128;
      const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
      const int lim = u.len - p.n + 1 + (wp.row0 + me) / p.G;  // tokens that row `me` sees
      float m = kNegInf, l = 0.f;
      for (int k = 0; k < n; ++k) {
        const int at = it + k, buf = at & 1, first = t0 + k * Gm::KEYS;
        const int t = first + me;
        Cell cell = {0, 0, false};
        size_t place = 0;
        float before = 0.f;
        if (SUMS && t < t1) {
          cell = token_cell<PAGED>(p.page_table, p.max_pages, p.page_size, p.num_pages, u.b, t);
          place = ((size_t)cell.slab * p.Hkv + u.h) * (PAGED ? p.page_size : p.ctx) + cell.at;
          if (wp.prior && cell.good) before = load_dependent(wp.prior + place);
        }
        if (!__all_sync(0xffffffffu, wait(Gm::BAR_SF + buf, at >> 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float* ks = reinterpret_cast<const float*>(smem + Gm::OFF_KS) + (at & 7) * Gm::KEYS;
        const int end = min(t1, SUMS ? t1 : lim) - first;  // keys of the tile that the row sees
        const float mine = SUMS ? ks[me] : 0.f;
        // SUMS: the first row that sees the token (an early one's product with G could pass 32 bits below 0)
        const int from = SUMS ? max(t - (u.len - p.n), 0) * p.G - wp.row0 : 0;
        const bool edge = SUMS ? __any_sync(0xffffffffu, from > 0) : __any_sync(0xffffffffu, end < Gm::KEYS);
        float w = 0.f;
#pragma unroll 1
        for (int c0 = 0; c0 < (SUMS ? wp.rows : Gm::KEYS); c0 += 32) {
          uint32_t r[32];
          tmem_ld32(tmem + lane_addr + buf * 128 + c0, r);
          tmem_ld_wait();
          if constexpr (SUMS) {
            const float4* f = reinterpret_cast<const float4*>(smem + Gm::OFF_F) + c0 / 2;
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 mine2 = make_float2(mine, mine);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float4 g = f[i];
              float2 y = fma_f32x2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), mine2,
                                   make_float2(g.x, g.y));
              float2 part = make_float2(g.z, g.w);
              if (edge) {  // a row that does not see the token gives it nothing, not even its NaN
                const bool a = c0 + 2 * i >= from, b = c0 + 2 * i + 1 >= from;
                y = make_float2(a ? y.x : kNegInf, b ? y.y : kNegInf);
                part = make_float2(a ? part.x : 0.f, b ? part.y : 0.f);
              }
              acc[i & 1] = fma_f32x2(make_float2(exp2_approx(y.x), exp2_approx(y.y)), part, acc[i & 1]);
            }
            w += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
          } else {
            const float4* s4 = reinterpret_cast<const float4*>(ks + c0);
            float2 y[16];  // the scores times their scales (into the exponents' fma they need more registers than there are)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float4 g = make_float4(p.scale_log2, p.scale_log2, p.scale_log2, p.scale_log2);
              if constexpr (INT8) g = s4[i];
              const float2 zero = make_float2(0.f, 0.f);
              y[2 * i] =
                  fma_f32x2(make_float2(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])), make_float2(g.x, g.y), zero);
              y[2 * i + 1] = fma_f32x2(make_float2(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])),
                                       make_float2(g.z, g.w), zero);
              if (edge) {
                const int left = end - c0 - 4 * i;
                y[2 * i].x = left > 0 ? y[2 * i].x : kNegInf;
                y[2 * i].y = left > 1 ? y[2 * i].y : kNegInf;
                y[2 * i + 1].x = left > 2 ? y[2 * i + 1].x : kNegInf;
                y[2 * i + 1].y = left > 3 ? y[2 * i + 1].y : kNegInf;
              }
            }
            auto total = [&]() {
              const float mu = m == kNegInf ? 0.f : m;
              const float2 mu2 = make_float2(-mu, -mu);
              float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 z = add_f32x2(y[i], mu2);
                acc[i & 1] = add_f32x2(acc[i & 1], make_float2(exp2_approx(z.x), exp2_approx(z.y)));
              }
              return (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
            };
            // against the m so far; a row that has seen no key yet, or whose weights sum past 2^14, raises it (the
            // maximum of every 32 first: 53.7 us instead of 51.6 for 32 tokens x 32 heads over 32768 int8 keys)
            float sum = total();
            if (m == kNegInf || !(sum <= 16384.f)) {
              float2 top = make_float2(m, m);
#pragma unroll
              for (int i = 0; i < 16; ++i) top = make_float2(fmaxf(top.x, y[i].x), fmaxf(top.y, y[i].y));
              const float to = fmaxf(top.x, top.y);
              if (to > m) {
                l *= exp2_approx(m - to);
                m = to;
              }
              sum = total();
            }
            l += sum;
          }
        }
        tc_fence_before();
        mbar_arrive(bar(Gm::BAR_SE + buf));
        if (SUMS && t < t1 && cell.good) wp.out[place] = wp.prior ? fmaf(wp.decay, before, w) : w;
      }
      if (!SUMS && ok) p.part_ml[((size_t)u.id + blockIdx.x) * Gm::ROWS + me] = make_float2(m, l);
    }
    ok = !__syncthreads_or(!ok);
    it += n;
    x += tiles64;
    if (x < x1) {
      u = walk.next(u);
      j = 0;
    }
  }
  if (warp == 8) {
    // before the tensor memory is freed, every product issued must have completed
    if (issued && elect_one()) {
      tc_commit(bar(Gm::BAR_FIN));
      const uint64_t at = globaltimer_ns();
      while (!mbar_try_wait(bar(Gm::BAR_FIN), 0) && globaltimer_ns() - at < wp.timeout_ns) {
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

}  // namespace da
