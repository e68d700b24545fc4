// The shared prefix's part of prefix attention on the 5th-generation tensor cores: every
// query row of the batch against the same keys and values, without a mask but for rows whose
// sequence ends inside the prefix.
//
// The rows of a KV head are those of all B q_len tokens times its G query heads, so a batch
// turns the prefix into two dense products,
//   S = Q K^T,  O = 2^(S - m) V,
// (a weight of 0 times a value that is not finite is NaN: rows that do not see all of the prefix and come out so are
// computed by themselves in seg_merge_prefix_kernel)
// 4 D operations a (row, key) and D * 4 bytes a key once a block of rows: bound by the bytes
// up to about 128 rows, then by the tensor cores and, beside them, one exponential a (row,
// key).  The engine is that of latent_prefill.cuh: a CTA owns up to two tiles of 128 rows (one
// at D = 256), whose rows are the lanes of tensor memory; each has a softmax warpgroup, one
// thread a row; with two, the tensor cores run one tile's products while the other's softmax
// works:
//   P_A V_j, S_A = Q_A K_{j+1}^T, P_B V_j, S_B = Q_B K_{j+1}^T;
// with one, S has two buffers and S_{j+1} is computed ahead of P_j V_j.  Tensor memory: two S
// of 128 columns (64 at D = 256) and the O (D columns each).  K and V come through one ring
// of granules, a tile's keys or values each, freed by their last product (16 KB ones at D >= 128 cost the
// producers one more chain of wait, look-up and boxes a 16 KB: 62.6 us a call of 64 x (16384 + <= 2048)
// tokens, 64/8 heads of 128, instead of 60.1; 52.9 instead of 48.8 at 16 x 4 rows of 24/4 heads of 256 after
// 8192).  A tile is 128 keys, 64 at D = 256: a ring of 160 KB holds one and a quarter of 128 keys there, and
// K_{j+1} next to V_j leaves hardly any of it to loads in flight.  Multicast of the keys to clusters of the row
// blocks that share them did not help (2.0 -> 2.3 us a tile, D = 128): their loads are not
// bound by L2's rate.
//
// The key tiles are cut into `splits` parts so that parts x row blocks x heads fill the
// card once; every part leaves (O, m, l) unnormalised in fp32 and seg_merge_prefix_kernel
// joins them with the rests'.
//
// Measured: 512 rows x 16384 keys x 8 heads, D = 128, pages of 16: 26 us, 1.4 us a tile of 128 keys x 256 rows (96% of
// the tensor rate), 4 us of start and 2 of partials' stores; 384 rows x 8192 x 4, D = 256: 18 us, 0.9 us a tile
// of 64 x 128 (0.7 at the tensor rate).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "device_error.cuh"
#include "ptx.cuh"
#include "seg_kernel.cuh"
#include "tc05.cuh"

namespace da {

struct PrefixTcParams {
  CUtensorMap tm_k, tm_v;   // [pages][Hkv][D / 64][rows of a page][64]; boxes of 2^rk_log2, 2^rv_log2 rows and 64 elements
  const __nv_bfloat16* q;   // [B, n, Hq, D]
  const int* seq_lens;      // or null: cap
  const int* prefix_table;  // null: the prefix is one page
  float* o;                 // [splits][Hkv][B n G][D]
  float2* ml;               // [splits][Hkv][B n G]: m in log2 units, l
  int B, n, Hq, Hkv, G;
  int P, cap;
  int page_size, num_pages;
  int rk_log2, rv_log2;
  int splits, row_blocks;
  float scale_log2;
  unsigned long long timeout_ns;
};

template <int D>
struct PrefixTcGeo {
  static constexpr int M = 128, BK = D == 256 ? 64 : 128;
  static constexpr int NQT = D <= 128 ? 2 : 1;  // query tiles a CTA
  static constexpr int ROWS = NQT * M;
  static constexpr int NSUB = D / 64;           // 64-element columns
  static constexpr int GB = D >= 128 ? 32768 : 16384;  // bytes a granule
  static constexpr int KSUB = GB / (BK * 128);  // 64-element columns of a K granule
  static constexpr int VKEYS = GB / (2 * D);    // keys of a V granule
  static constexpr int NKG = NSUB / KSUB, NVG = BK / VKEYS, PER = NKG + NVG;
  static constexpr int QT_BYTES = M * D * 2;
  static constexpr int OFF_G = NQT * QT_BYTES;
  static constexpr int NG_FIT = (227 * 1024 - 2048 - OFF_G) / GB;
  static constexpr int NG = NG_FIT < 12 ? NG_FIT : 12;
  static constexpr int OFF_BAR = OFF_G + NG * GB;
  static constexpr int BAR_FULL = 0, BAR_EMPTY = NG, BAR_S = 2 * NG, BAR_P = BAR_S + 2, BAR_O = BAR_P + 2,
                       BAR_FIN = BAR_O + 2, NBAR = BAR_FIN + 1;
  static constexpr int OFF_MISC = OFF_BAR + (NBAR + 1) / 2 * 16;  // tensor memory base, abort flag
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static constexpr int TCOL_O = 2 * BK;  // S buffer i at i BK, O of tile t at TCOL_O + t D
  static constexpr uint32_t TMEM_COLS = TCOL_O + NQT * D <= 256 ? 256u : 512u;
  static constexpr int NTHREADS = 128 + 128 * NQT;
  static constexpr int REG_LOW = 120, REG_HIGH = 192;  // after the split of the two-tile form
  static constexpr int REG_POOL_NEEDED = 128 * REG_LOW + 128 * NQT * REG_HIGH;
  static_assert(NG >= PER + (NQT == 1 ? 1 : NVG) && SMEM <= 227 * 1024, "the ring holds what the products hold at once");
  static_assert(TCOL_O + NQT * D <= 512, "tensor memory");
};

template <int N>
__device__ __forceinline__ void prefix_setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void prefix_setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D>
__global__ void __launch_bounds__(PrefixTcGeo<D>::NTHREADS, 1) prefix_tc_kernel(const __grid_constant__ PrefixTcParams p) {
  using Gm = PrefixTcGeo<D>;
  constexpr int BK = Gm::BK, M = Gm::M, NQT = Gm::NQT;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  auto bar = [&](int i) -> uint32_t { return sbase + Gm::OFF_BAR + 8 * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Gm::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // work: the row blocks of a (head, part) side by side, as they read the same keys
  const int rb = blockIdx.x % p.row_blocks, hs = blockIdx.x / p.row_blocks;
  const int s = hs % p.splits, h = hs / p.splits;
  const int T = (p.P + BK - 1) / BK;
  const int j0 = (int)((long long)T * s / p.splits), ntiles = (int)((long long)T * (s + 1) / p.splits) - j0;
  const int all_rows = p.B * p.n * p.G;
  const int row0 = rb * Gm::ROWS, nrows = min(Gm::ROWS, all_rows - row0);
  const int nqt = NQT == 2 && nrows > M ? 2 : 1;  // query tiles with rows

  if (threadIdx.x == 0) {
    for (int i = 0; i < Gm::NG; ++i) {
      mbar_init(bar(Gm::BAR_FULL + i), 1);
      mbar_init(bar(Gm::BAR_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(Gm::BAR_S + i), 1);
      mbar_init(bar(Gm::BAR_P + i), 4);  // one arrival a warp
      mbar_init(bar(Gm::BAR_O + i), 1);
    }
    mbar_init(bar(Gm::BAR_FIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&p.tm_k);
    prefetch_tensormap(&p.tm_v);
  }
  // Tensor memory is taken after the wait and before the next kernel may start: none waits for another
  // while it holds some that the other still has to take.
  pdl_wait_primary();
  if (warp == 1) {
    tmem_alloc(sbase + Gm::OFF_MISC, Gm::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // the rests' kernel may start as soon as SMs are free: what it reads was written before this
  // kernel's wait ended, and it waits for this kernel at its end
  pdl_launch_dependents();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Gm::OFF_MISC);
  auto wait = [&](int i, int phase) { return wait_bounded(bar(i), (uint32_t)(phase & 1), abort_flag, p.timeout_ns); };
  // granule g of this CTA's tile j: K columns 0 .. NKG - 1, then V
  auto slot_of = [&](int j, int g) { return (j * Gm::PER + g) % Gm::NG; };
  auto fill_of = [&](int j, int g) { return (j * Gm::PER + g) / Gm::NG; };
  auto addr_of = [&](int j, int g) { return sbase + Gm::OFF_G + (uint32_t)(slot_of(j, g) * Gm::GB); };

  // query rows, [tile][D / 64][128][64] with the 128-byte swizzle, zeros past the last; by the warps
  // that need them, while the first keys load, all copies in flight at once
  auto stage_queries = [&](int me) {
    constexpr int CH = D / 8, N = 32 + 128 * NQT, STEP = N / CH;  // a thread's chunk of every STEP-th row
    static_assert(N % CH == 0, "");
    const int ch = me % CH, more = STEP / p.G, step_g = STEP - more * p.G;
    const uint32_t column = sbase + (ch / 8) * (M * 128);
    int token = (row0 + me / CH) / p.G, g = row0 + me / CH - token * p.G;
    const __nv_bfloat16* from = p.q + (size_t)h * p.G * D + ch * 8;
#pragma unroll 4
    for (int rr = me / CH; rr < nqt * M; rr += STEP) {
      const bool is = rr < nrows;
      cp_async16(column + (rr / M) * Gm::QT_BYTES + swz<128>(rr % M, ch % 8),
                 is ? from + ((size_t)token * p.Hq + g) * D : p.q, is);
      token += more;
      g += step_g;
      if (g >= p.G) {
        g -= p.G;
        ++token;
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
    fence_proxy_async_smem();
    named_bar_sync(1, N);
  };

  if (warp < 4) {
    if constexpr (NQT == 2) prefix_setmaxnreg_dec<Gm::REG_LOW>();
    if (warp != 1) {
      // ---- producers: granules in the order of the products, a granule's boxes dealt to the lanes
      // of three warps (a page of 16 tokens is 2 KB of each column, and a warp issues its boxes one
      // after another: 3.4 us a tile of 32 with one warp, 2.6 with three, D = 128).  Boxes wholly
      // past the prefix are not loaded.  No warp falls a round of the ring behind: a granule is not
      // full, and so not freed, without every warp's boxes.
      const int pid = warp == 0 ? 0 : warp - 1;
      bool ok = true;
      int last = -1;
      // lane l < BK / 16: the page of the tile's keys from 16 l on and their row in it, looked up a
      // tile ahead
      int row_ahead = 0;
      auto page_of = [&](int j) {
        const int tok = (j0 + j) * BK + 16 * lane;
        row_ahead = tok;
        if (!p.prefix_table || lane >= BK / 16 || j >= ntiles || tok >= p.P) return 0;
        const int col = tok / p.page_size;
        row_ahead = tok - col * p.page_size;
        const int page = load_dependent(p.prefix_table + col);
        if ((unsigned)page < (unsigned)p.num_pages) return page;
        atomicOr(&g_error_word, 4u);
        return 0;
      };
      int ahead = page_of(0);
      for (int j = 0; j < ntiles && ok; ++j) {
        const int t0 = (j0 + j) * BK, pages = ahead, page_rows = row_ahead;
        ahead = page_of(j + 1);
        const bool whole = t0 + BK <= p.P;
#pragma unroll 1
        for (int g = 0; g < Gm::PER; ++g) {
          const int fill = fill_of(j, g), slot = slot_of(j, g);
          const bool is_k = g < Gm::NKG;
          const int shift = is_k ? p.rk_log2 : p.rv_log2, keys = is_k ? BK : Gm::VKEYS;
          const int first = is_k ? 0 : (g - Gm::NKG) * Gm::VKEYS;  // key of the tile
          const int live = whole ? keys : max(0, min(keys, p.P - t0 - first));
          const int boxes = (live + (1 << shift) - 1) >> shift;  // a column
          const int box = 3 * lane + pid;
          int sub = 0, bx = box;  // the column of the granule, and the box of it
#pragma unroll
          for (int c = 1; c < Gm::NSUB; ++c)
            if (bx >= boxes && sub + 1 < (is_k ? Gm::KSUB : Gm::NSUB)) {
              bx -= boxes;
              ++sub;
            }
          const int at = (first >> 4) + (bx << shift >> 4);
          const int page = __shfl_sync(0xffffffffu, pages, at & 31), row = __shfl_sync(0xffffffffu, page_rows, at & 31);
          const int n = boxes * (is_k ? Gm::KSUB : Gm::NSUB);
          if (fill > 0 && !(ok = __all_sync(0xffffffffu, wait(Gm::BAR_EMPTY + slot, fill - 1)))) break;
          const uint32_t full = bar(Gm::BAR_FULL + slot);
          if (pid == 0 && lane == 0) {
            if (n > 0)
              mbar_arrive_expect_tx(full, (uint32_t)(n << shift) * 128u);
            else
              mbar_arrive(full);
          }
          if (bx < boxes)
            tma_load_5d(addr_of(j, g) + (uint32_t)(sub * keys * 128 + (bx << shift) * 128), is_k ? &p.tm_k : &p.tm_v, full, 0,
                        row, is_k ? g * Gm::KSUB + sub : sub, h, page);
          last = j * Gm::PER + g;
        }
      }
      if (*abort_flag && lane == 0) {  // copies in flight land before the CTA exits
        const uint64_t at = globaltimer_ns();
        for (int m = last; m >= 0 && m > last - Gm::NG; --m)
          while (!mbar_try_wait(bar(Gm::BAR_FULL + m % Gm::NG), (uint32_t)((m / Gm::NG) & 1)) &&
                 globaltimer_ns() - at < p.timeout_ns) {
          }
      }
      __syncwarp();
    } else {
      // ---- MMA issue (one lane); the warp zeroes V rows past the prefix
      stage_queries(threadIdx.x - 32);
      constexpr uint32_t id_s = tc_idesc_bf16(M, BK, false, false);
      constexpr uint32_t id_o = tc_idesc_bf16(M, D, false, true);
      auto wait_all = [&](int i, int phase) { return __all_sync(0xffffffffu, wait(i, phase)) != 0; };
      auto landed = [&](int j, int g0, int g1) {
        bool there = true;
        for (int g = g0; g < g1; ++g) there = wait(Gm::BAR_FULL + slot_of(j, g), fill_of(j, g)) && there;
        return __all_sync(0xffffffffu, there) != 0;
      };
      // one thread: S buffer sb = Q_t K_j^T; the granules are freed after the last query tile
      auto issue_qk = [&](int t, int j, int sb) {
#pragma unroll
        for (int g = 0; g < Gm::NKG; ++g) {
          const uint64_t da = tc_sdesc(sbase + t * Gm::QT_BYTES + g * Gm::KSUB * (M * 128), 16, 1024, kTcSwizzle128B);
          const uint64_t db = tc_sdesc(addr_of(j, g), 16, 1024, kTcSwizzle128B);
#pragma unroll
          for (int i = 0; i < 4 * Gm::KSUB; ++i)
            tc_mma_ss(tmem + sb * BK, da + (i / 4) * (M * 128 / 16) + 2 * (i % 4), db + (i / 4) * (BK * 128 / 16) + 2 * (i % 4),
                      id_s, g > 0 || i > 0);
          if (t == nqt - 1) tc_commit(bar(Gm::BAR_EMPTY + slot_of(j, g)));
        }
        tc_commit(bar(Gm::BAR_S + sb));
      };
      // one thread: O_t += P (S buffer sb) V_j
      auto issue_pv = [&](int t, int j, int sb) {
#pragma unroll
        for (int g = 0; g < Gm::NVG; ++g) {
          const uint64_t db = tc_sdesc(addr_of(j, Gm::NKG + g), Gm::VKEYS * 128, 1024, kTcSwizzle128B);
#pragma unroll
          for (int i = 0; i < Gm::VKEYS / 16; ++i)
            tc_mma_ts(tmem + Gm::TCOL_O + t * D, tmem + sb * BK + 8 * (g * (Gm::VKEYS / 16) + i), db + i * 128, id_o,
                      j > 0 || g > 0 || i > 0);
          if (t == nqt - 1) tc_commit(bar(Gm::BAR_EMPTY + slot_of(j, Gm::NKG + g)));
        }
        // with two tiles O_t is waited for once, at the end; with one, every other P V completes the
        // same barrier, so that a wait for either is never a phase behind
        if (NQT == 1)
          tc_commit(bar(Gm::BAR_O + (j & 1)));
        else if (j + 1 == ntiles)
          tc_commit(bar(Gm::BAR_O + t));
      };
      // V rows at or past the prefix may hold anything (0 * NaN would poison O): zero them
      auto zero_tail = [&](int j) {
        for (int g = 0; g < Gm::NVG; ++g) {
          const int r0 = max(0, p.P - ((j0 + j) * BK + g * Gm::VKEYS));
          uint8_t* vs = smem + Gm::OFF_G + slot_of(j, Gm::NKG + g) * Gm::GB;
          for (int e = r0 * 8 + lane; e < Gm::VKEYS * 8; e += 32)
            for (int c = 0; c < Gm::NSUB; ++c)
              *reinterpret_cast<uint4*>(vs + c * (Gm::VKEYS * 128) + swz<128>(e / 8, e % 8)) =
                  make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
      };
      bool ok = ntiles > 0 && landed(0, 0, Gm::NKG);
      const bool any = ok;
      if (ok && elect_one()) {
        tc_fence_after();
        for (int t = 0; t < nqt; ++t) issue_qk(t, 0, t);
      }
      __syncwarp();
      for (int j = 0; j < ntiles && ok; ++j) {
        const bool more = j + 1 < ntiles;
        if constexpr (NQT == 2) {
          if (!(ok = landed(j, Gm::NKG, Gm::PER))) break;
          if ((j0 + j + 1) * BK > p.P) zero_tail(j);
          if (!(ok = wait_all(Gm::BAR_P, j))) break;
          if (elect_one()) {
            tc_fence_after();
            issue_pv(0, j, 0);
          }
          __syncwarp();
          if (more) {
            if (!(ok = landed(j + 1, 0, Gm::NKG))) break;
            if (elect_one()) {
              tc_fence_after();
              issue_qk(0, j + 1, 0);
            }
            __syncwarp();
          }
          if (nqt == 2) {
            if (!(ok = wait_all(Gm::BAR_P + 1, j))) break;
            if (elect_one()) {
              tc_fence_after();
              issue_pv(1, j, 1);
              if (more) issue_qk(1, j + 1, 1);
            }
            __syncwarp();
          }
        } else {
          if (more) {
            if (!(ok = landed(j + 1, 0, Gm::NKG))) break;
            if (elect_one()) {
              tc_fence_after();
              issue_qk(0, j + 1, (j + 1) & 1);
            }
            __syncwarp();
          }
          if (!(ok = landed(j, Gm::NKG, Gm::PER))) break;
          if ((j0 + j + 1) * BK > p.P) zero_tail(j);
          if (!(ok = wait_all(Gm::BAR_P + (j & 1), j >> 1))) break;
          if (elect_one()) {
            tc_fence_after();
            issue_pv(0, j, j & 1);
          }
          __syncwarp();
        }
      }
      // before the tensor memory is freed, every MMA issued must have completed
      if (any && elect_one()) {
        tc_commit(bar(Gm::BAR_FIN));
        const uint64_t at = globaltimer_ns();
        while (!mbar_try_wait(bar(Gm::BAR_FIN), 0) && globaltimer_ns() - at < p.timeout_ns) {
        }
      }
      __syncwarp();
    }
  } else {
    // ---- softmax of query tile qt and its partial: one thread per row (tensor memory lane)
    if constexpr (NQT == 2) prefix_setmaxnreg_inc<Gm::REG_HIGH>();
    stage_queries(threadIdx.x - 96);
    const int qt = (warp >> 2) - 1;
    const int row = qt * M + lane + 32 * (warp & 3);
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_addr = tmem + lane_addr + Gm::TCOL_O + qt * D;
    const bool has_row = row < nrows;
    int lim = p.P;  // keys this row sees
    if (has_row) {
      const int token = (row0 + row) / p.G, b = token / p.n;
      lim = max(0, min(p.P, seg_len(p.seq_lens, b, p.cap) - p.n + 1 + (token - b * p.n)));
    }
    const int lim_first = __reduce_min_sync(0xffffffffu, lim);  // keys every row of the warp sees
    const bool fold = p.scale_log2 > 0.f;  // a positive scale goes into the exponent's fma
    const float sc = fold ? p.scale_log2 : 1.f;
    float m = kNegInf, l = 0.f;
    bool ok = qt < nqt;
    for (int j = 0; j < ntiles && ok; ++j) {
      const int sb = NQT == 2 ? qt : j & 1;
      const uint32_t s_addr = tmem + lane_addr + sb * BK;
      ok = __all_sync(0xffffffffu, wait(Gm::BAR_S + sb, NQT == 2 ? j : j >> 1));
      if (!ok) break;
      tc_fence_after();
      float x[BK];
      {
        uint32_t r[BK];
#pragma unroll
        for (int c0 = 0; c0 < BK; c0 += 32) tmem_ld32(s_addr + c0, *reinterpret_cast<uint32_t(*)[32]>(r + c0));
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < BK; ++i) x[i] = __uint_as_float(r[i]);
      }
      if (!fold) {
#pragma unroll
        for (int i = 0; i < BK; ++i) x[i] *= p.scale_log2;
      }
      if ((j0 + j + 1) * BK > lim_first) {
        const int left = lim - (j0 + j) * BK;
#pragma unroll
        for (int i = 0; i < BK; ++i) x[i] = i < left ? x[i] : kNegInf;
      }
      // P = exp2(x sc - mu) as bf16 pairs over the first half of the S buffer; the sum of the weights
      auto weights = [&](float mu) {
        float2 sk[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) sk[k] = make_float2(0.f, 0.f);
        const float2 sc2 = make_float2(sc, sc), mu2 = make_float2(-mu, -mu);
#pragma unroll
        for (int c0 = 0; c0 < BK / 2; c0 += 32) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 y = fma_f32x2(make_float2(x[2 * (c0 + i)], x[2 * (c0 + i) + 1]), sc2, mu2);
            const float2 e = make_float2(exp2_approx(y.x), exp2_approx(y.y));
            sk[i & 3] = add_f32x2(sk[i & 3], e);
            pk[i] = pack_bf16x2(e.x, e.y);
          }
          tmem_st32(s_addr + c0, pk);
        }
        const float2 t = add_f32x2(add_f32x2(sk[0], sk[1]), add_f32x2(sk[2], sk[3]));
        return t.x + t.y;
      };
      // The weights are first taken against the current m; only a row that has seen no key
      // yet, or whose weights sum past 2^14, takes its maximum and raises m to it.  The stores
      // in weights() are the whole warp's, so every call is warp-uniform.
      const bool have = __any_sync(0xffffffffu, m != kNegInf);
      float sum = 0.f;
      if (have) sum = weights(m == kNegInf ? 0.f : m);
      const bool need = m == kNegInf || !(sum <= 16384.f);
      float mx = kNegInf;
      if (need) {
        float mk[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mk[k] = x[k];
#pragma unroll
        for (int i = 8; i < BK; ++i) mk[i & 7] = fmaxf(mk[i & 7], x[i]);
        mx = fmaxf(fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3])), fmaxf(fmaxf(mk[4], mk[5]), fmaxf(mk[6], mk[7])));
        mx = fold ? mx * p.scale_log2 : mx;
      }
      const bool raise = need && mx > m;
      const float m_new = raise ? mx : m;
      const float alpha = raise && m != kNegInf ? exp2_approx(m - m_new) : raise ? 0.f : 1.f;
      if (__any_sync(0xffffffffu, raise && m != kNegInf) && j > 0) {
        // O holds the P V of the tiles before.  Two query tiles: S of tile j was issued after P V
        // of tile j - 1, and its commit covers every MMA before it.  One: wait for that P V
        if constexpr (NQT == 1) {
          if (!(ok = __all_sync(0xffffffffu, wait(Gm::BAR_O + ((j - 1) & 1), (j - 1) >> 1)))) break;
          tc_fence_after();
        }
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(o_addr + c0, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st32(o_addr + c0, o);
        }
        tmem_st_wait();
      }
      m = m_new;
      if (!have || __any_sync(0xffffffffu, raise)) sum = weights(m == kNegInf ? 0.f : m);
      l = l * alpha + sum;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Gm::BAR_P + sb));
    }
    if (ok && ntiles > 0)
      ok = __all_sync(0xffffffffu, NQT == 2 ? wait(Gm::BAR_O + qt, 0)
                                            : wait(Gm::BAR_O + ((ntiles - 1) & 1), (ntiles - 1) >> 1));
    if (qt < nqt) {
      tc_fence_after();
      const size_t at = ((size_t)s * p.Hkv + h) * all_rows + row0 + row;
      if (has_row) p.ml[at] = make_float2(m, ok ? l : 0.f);
// O goes out through the queries' place, which the products have done with, so that a store instruction
      // writes 4 rows of 128 bytes (16 bytes of 32 rows: 4.9 us of the 29.6 that 384 rows x 8192 keys, D = 256, take)
      const uint32_t scratch = sbase + qt * Gm::QT_BYTES + (warp & 3) * (Gm::QT_BYTES / 4);
      const int first = qt * M + 32 * (warp & 3);
      float* o = p.o + (((size_t)s * p.Hkv + h) * all_rows + row0 + first) * D;
#pragma unroll 1
      for (int c0 = 0; c0 < D && ok && ntiles > 0; c0 += 32) {  // (l is 0 with no tile, and nothing else read)
        uint32_t r[32];
        tmem_ld32(o_addr + c0, r);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(scratch + lane * 128 + ((k ^ (lane & 7)) << 4)),
                       "r"(r[4 * k]), "r"(r[4 * k + 1]), "r"(r[4 * k + 2]), "r"(r[4 * k + 3])
                       : "memory");
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = 4 * i + lane / 8, c = lane & 7;
          uint4 v;
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "r"(scratch + rr * 128 + ((c ^ (rr & 7)) << 4)));
          if (first + rr < nrows) *reinterpret_cast<uint4*>(o + (size_t)rr * D + c0 + 4 * c) = v;
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Gm::TMEM_COLS);
  }
}

}  // namespace da
