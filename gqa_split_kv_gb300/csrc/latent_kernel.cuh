// Attention over a cache of one shared latent vector a token (the absorbed form), for
// the last q_len tokens of every sequence, on the 5th-generation tensor cores.
//
//   s_t = scale <q, c_t>,   out = sum_t softmax(s)_t c_t[0 : R],   c_t of W = R + 64
//
// All H heads of a token share every cache row, so the rows of one product are the
// (token, head) pairs of a sequence, and the cache is both K and V: a row is read from
// HBM once and used twice from shared memory.  2 N (2 R + 64) operations a token and
// 2 (R + 64) bytes: N = 16 rows are 30 operations a byte, far on the HBM side of this
// card's 294; 64 rows 121; 128 rows 242.
//
// Both products are taken transposed, the cache as the left operand:
//   S^T (64 tokens x N rows)   = C (64 x W, K-major) Q^T,
//   O^T (R x N rows)          += C[:, 0:R]^T (128 latents a block x 64 tokens, MN-major from
//                                the same shared memory) P^T.
// The accumulator of R latents is then R / 128 blocks of N columns of tensor memory
// (256 of 512 columns at R = 512, N = 64), where R columns for the rows as lanes would
// leave no room for S, and a few rows cost no more than they are: N is 16, 32 or 64.  64
// tokens a tile, not 128: with Q (72 KB at N = 64) in shared memory a 128-token tile
// (144 KB) could not be double-buffered.
//
// A tile is R / 128 units of 16 KB ([2][64 tokens][64 elements], 128-byte swizzle) and
// the rotated part (8 KB) in a ring of its own; a unit is freed by its own P^T product.  The
// ring has to hold two whole tiles: with one unit less (7 at N = 64) the last unit of a
// tile waits for the first product of the tile before it, and a tile takes that
// latency (0.8 us) and a load's (1.5 us) instead of half of it: 2.27 us a tile with 7 units,
// 1.96 with 8.  So at N = 64, R = 512 the plan's arrays share the ring's memory, each
// CTA's pieces are listed once, and P^T has one buffer.
//
// Softmax.  S comes back as the fragment of a 16 x 8 warp MMA: thread t of warp w holds
// tokens 16 w + t / 4 and 8 further on, N / 4 rows of each; P^T is stored with transposing
// stmatrix, 16 bytes of tokens a row.  The maximum of a row is over tokens, so over
// lanes and warps; but any reference m near it gives the same quotient, so m stays as it
// is until a score passes it by more than 24 (log2): one vote a tile instead of a
// reduction.  Weights then stay under 2^24, and their sums far inside fp32.  l sums the
// weights as rounded to bf16 for the product, so a row with one heavy token is exact.
//
// Split.  The plan of plan.cuh, with (sequence, row tile) segments and one range of the
// line per SM.  A range holds at most two pieces of segments that other ranges share, so
// two slots of N rows per range hold every partial (152 ranges: 40 MB at N = 64, R =
// 512), whatever the batch; latent_combine_kernel merges them.
//
// Warps: 0 and 3 issue the copies (Q and even units; odd units and the rotated part), 1
// the S products, 2 the O products, from 4 on softmax and epilogue, a warpgroup per 32
// rows.  The issuing lane is chosen by elect.sync: behind a lane compare the compiler
// guards every MMA, 45 cycles each, behind elect.sync 23, which at N <= 32 is less than the
// tensor core takes (batch below: 57.8 -> 47.9 us).  Waits are bounded as in prefill_tc.cuh.
//
// Bound and measured (bf16, R = 512).  16 sequences up to 8192 tokens, 128 heads: 41.0
// us, where HBM needs 12.3 and the tensor cores 9.6; 64 sequences of 1 to 32768 tokens, 64
// heads: 61.6 us, HBM 36.0; one sequence of 4096 tokens, 16 heads: 10.8 us.  A tile of 64
// rows takes 1.85 us: the round through its two ring slots (load 1.5 us, S 0.6, softmax
// 0.5, O 0.4, overlapping by units), not HBM (85 MB of it are read once, by the other row
// tile from L2), with the tensor cores 35% busy.  Around the tiles: 5 us to the first
// tile's products (launch, plan, Q and the first load), 2.4 us for the partials, and the merge,
// 3 to 6 us, whose 22 MB come from L2.  Tried and dropped: prefetching 4 tiles ahead into
// L2 (2.5 us a tile), and pairs of CTAs that share a tile by multicast (1.65 us a tile but 2
// us more at the start and end: 49.4 against 49.2 us).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "device_error.cuh"
#include "plan.cuh"
#include "ptx.cuh"
#include "tc05.cuh"

namespace da {

struct LatentParams {
  CUtensorMap tm_q;     // [B][W / 64][rows][64], boxes of N rows and every column
  CUtensorMap tm_unit;  // cache [slab][W / 64][tokens][64], boxes of 16, 32 or 64 tokens and 1 or 2 columns
  CUtensorMap tm_pe;    // the same, 1 column
  const int* seq_lens;
  const int* page_table;
  float* part_acc;      // [2 ranges][N][R]
  float2* part_ml;      // [2 ranges][N], m in log2 units
  int4* pieces;         // [ranges + B U]: the ranges' pieces past the first LatentGeo::PCAP
  __nv_bfloat16* out;   // [B][rows][R]
  int B, H, q_len, rows, U;
  int ranges;           // ranges the line is cut into (at most)
  int max_len;
  int page_size, max_pages, num_pages, box_shift, page_shift;
  float scale_log2;
  unsigned long long timeout_ns;
};

// Line positions (16 tokens each) charged for a segment's fixed cost (64 sequences of 1 to
// 32768 tokens: 69.3 us with 4, 61.5 with 8, 63.1 with 12; 16 sequences 43.3, 42.5, 42.1).
constexpr int kLatentGap = 8;

// Sequence b's length, before the plan clamps it.
template <typename Params>
__device__ __forceinline__ auto latent_length(const Params& p) {
  return [&p](int b) { return p.seq_lens ? load_dependent(p.seq_lens + b) : p.max_len; };
}

// The cut of the line into `ranges` equal ranges.
__device__ __forceinline__ Plan latent_plan(int B, int U, int ranges, const int* P) {
  Plan pl;
  pl.U = U;
  pl.S = 2;  // pieces are walked range by range
  pl.gap = kLatentGap;
  pl.NB = U * P[B];
  pl.q = (pl.NB + ranges - 1) / ranges;
  pl.q = (pl.q + kRangeQuantum - 1) / kRangeQuantum * kRangeQuantum;
  if (pl.q < kRangeQuantum) pl.q = kRangeQuantum;
  pl.ranges = (pl.NB + pl.q - 1) / pl.q;
  return pl;
}

// Partial slot of piece j of a segment whose first block lies in range r0: a range's
// first segment may have begun before it, its last may go on after it.
__host__ __device__ __forceinline__ int latent_slot(int r0, int j) { return j == 0 ? 2 * r0 + 1 : 2 * (r0 + j); }

// A piece as the warps of a CTA read it: (sequence, first token, last token + 1, row tile
// and partial slot + 1, 0 for a segment of one piece).
__device__ __forceinline__ int4 latent_piece(const Piece& pc, int r) {
  return make_int4(pc.b, pc.t0, pc.t1, pc.u | (pc.npieces == 1 ? 0 : (latent_slot(r - pc.j, pc.j) + 1) << 8));
}

template <int R, int N>
struct LatentGeo {
  static constexpr int T = 64;               // tokens a tile
  static constexpr int NC = R / 64 + 1;      // 64-element columns of a cache row
  static constexpr int NU = R / 128;         // units a tile
  static constexpr int UNIT = 2 * T * 128, PE = T * 128;
  static constexpr int Q_BYTES = NC * N * 128, P_BYTES = N * 128;
  static constexpr int NPE = 2;
  // P^T has two buffers but where the second would cost the ring its second whole tile
  static constexpr int NP = R == 512 && N == 64 ? 1 : 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_P = OFF_Q + Q_BYTES;
  static constexpr int OFF_PE = OFF_P + NP * P_BYTES;
  static constexpr int OFF_U = OFF_PE + NPE * PE;
  static constexpr int SCRATCH = 2048;       // barriers, reductions, the first pieces
  static constexpr int NUNIT_FIT = (227 * 1024 - 1024 - OFF_U - SCRATCH) / UNIT;
  static constexpr int NUNIT = NUNIT_FIT < 12 ? NUNIT_FIT : 12;
  static constexpr int OFF_SCR = OFF_U + NUNIT * UNIT;
  // barriers
  static constexpr int B_UFULL = 0, B_UEMPTY = NUNIT, B_PEFULL = 2 * NUNIT, B_PEEMPTY = B_PEFULL + NPE,
                       B_QFULL = B_PEEMPTY + NPE, B_QEMPTY = B_QFULL + 1, B_S = B_QEMPTY + 1, B_P = B_S + 2,
                       B_PV = B_P + 2, B_OFREE = B_PV + 2, B_FIN = B_OFREE + 1, NBAR = B_FIN + 2;
  static constexpr int OFF_MISC = OFF_SCR + NBAR * 8;          // tensor memory base, abort flag, pieces
  static constexpr int PCAP = 8;                               // pieces kept in shared memory
  static constexpr int OFF_PC = (OFF_MISC + 16 + 15) / 16 * 16;
  static constexpr int OFF_RED = OFF_PC + PCAP * 16;           // [4][N] floats
  static constexpr int OFF_COL = OFF_RED + 4 * N * 4;          // [N] floats: factors of O's columns
  static constexpr int OFF_COLM = OFF_COL + N * 4;             // [N] floats: maxima at a piece's end
  static constexpr int SMEM = OFF_SCR + SCRATCH + 1024;
  // the plan's arrays lie in the ring until the first copy goes out
  static constexpr int MAX_BATCH = (NUNIT * UNIT / 4 - 2) / 2;
  static constexpr int TCOL_S = NU * N;      // O block i at i N, then two S buffers
  static constexpr int TCOLS = (NU + 2) * N;
  static constexpr uint32_t TMEM_COLS = TCOLS <= 64 ? 64u : TCOLS <= 128 ? 128u : TCOLS <= 256 ? 256u : 512u;
  static constexpr int NWG = N >= 32 ? 2 : 1;  // softmax warpgroups, N / NWG rows each
  static constexpr int NTHREADS = 128 + 128 * NWG;
  static_assert(OFF_COLM + N * 4 <= OFF_SCR + SCRATCH, "scratch");
  static_assert(R % 128 == 0 && N % 16 == 0 && TCOLS <= 512, "tensor memory");
  static_assert(NUNIT >= 2 * NU, "the ring holds two tiles");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int R, int N, bool PAGED>
__global__ void __launch_bounds__(LatentGeo<R, N>::NTHREADS, 1) latent_kernel(const __grid_constant__ LatentParams p) {
  using Gm = LatentGeo<R, N>;
  constexpr int T = Gm::T, NU = Gm::NU;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  auto bar = [&](int i) -> uint32_t { return sbase + Gm::OFF_SCR + 8 * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Gm::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < Gm::NUNIT; ++i) {
      mbar_init(bar(Gm::B_UFULL + i), 1);
      mbar_init(bar(Gm::B_UEMPTY + i), 1);
    }
    for (int i = 0; i < Gm::NPE; ++i) {
      mbar_init(bar(Gm::B_PEFULL + i), 1);
      mbar_init(bar(Gm::B_PEEMPTY + i), 1);
    }
    mbar_init(bar(Gm::B_QFULL), 1);
    mbar_init(bar(Gm::B_QEMPTY), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(Gm::B_S + i), 1);
      mbar_init(bar(Gm::B_P + i), 4 * Gm::NWG);  // one arrival a warp
      mbar_init(bar(Gm::B_PV + i), 1);
      mbar_init(bar(Gm::B_FIN + i), 1);
    }
    mbar_init(bar(Gm::B_OFREE), 4 * Gm::NWG);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&p.tm_q);
    prefetch_tensormap(&p.tm_unit);
    prefetch_tensormap(&p.tm_pe);
  }
  if (warp == 1) {
    tmem_alloc(sbase + Gm::OFF_MISC, Gm::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait_primary();  // (what precedes this call in the stream)
  {
    // this CTA's range of the line and its pieces
    int* lens = reinterpret_cast<int*>(smem + Gm::OFF_U);
    int* P = lens + p.B;
    build_plan_arrays(latent_length(p), p.B, p.max_len, kLatentGap, lens, P, 0, Gm::NTHREADS);
    if (threadIdx.x == 0) {
      const Plan pl = latent_plan(p.B, p.U, p.ranges, P);
      const int r = blockIdx.x;
      int count = 0, x = r * pl.q, xe = min(x + pl.q, pl.NB), first = -1;
      while (r < pl.ranges && x < xe) {
        Piece pc;
        x = piece_at(pl, lens, P, p.B, x, xe, r, pc);
        // a range's list begins after the ranges and segments before it
        if (first < 0) first = r + pc.u * p.B + pc.b;
        if (pc.t1 == pc.t0) continue;  // only a gap
        const int4 e = latent_piece(pc, r);
        if (count < Gm::PCAP)
          reinterpret_cast<int4*>(smem + Gm::OFF_PC)[count] = e;
        else
          p.pieces[first + count] = e;
        ++count;
      }
      *reinterpret_cast<int*>(smem + Gm::OFF_MISC + 8) = count;
      *reinterpret_cast<int*>(smem + Gm::OFF_MISC + 12) = first;
    }
  }
  fence_proxy_async_smem();  // the ring's next writes are copies
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Gm::OFF_MISC);
  const int npieces = *reinterpret_cast<volatile int*>(smem + Gm::OFF_MISC + 8);
  const int4* more = p.pieces + *reinterpret_cast<volatile int*>(smem + Gm::OFF_MISC + 12);
  pdl_launch_dependents();  // (after this CTA's own wait: the combine kernel reads seq_lens at once)

  struct {
    int b, t0, t1, u, slot;
  } pc;
  // piece i of this CTA
  auto take = [&](int i) {
    if (i >= npieces) return false;
    const int4 e = i < Gm::PCAP ? reinterpret_cast<const int4*>(smem + Gm::OFF_PC)[i] : more[i];
    pc.b = e.x;
    pc.t0 = e.y;
    pc.t1 = e.z;
    pc.u = e.w & 255;
    pc.slot = (e.w >> 8) - 1;  // -1: the segment's only piece
    return true;
  };
  int n = 0;      // tiles so far (over all pieces)
  int piece = 0;  // pieces so far
  auto wait = [&](int b, int phase) { return wait_bounded(bar(b), (uint32_t)(phase & 1), abort_flag, p.timeout_ns); };
  auto wait_all = [&](int b, int phase) { return __all_sync(0xffffffffu, wait(b, phase)) != 0; };

  if (warp == 0 || warp == 3) {
    // ---- producers.  Item k of a ring waits for the free of item k - slots by that slot's
    // phase; the slot's next phase is the free of item k itself, so the parity is never
    // a whole turn stale.
    if (lane == 0) {
      const bool second = warp == 3;
      bool ok = true;
      const int rsh = p.box_shift;
      while (ok && take(piece)) {
        if (!second) {
          if (piece > 0 && !(ok = wait(Gm::B_QEMPTY, piece - 1))) break;
          mbar_arrive_expect_tx(bar(Gm::B_QFULL), Gm::Q_BYTES);
          tma_load_4d(sbase + Gm::OFF_Q, &p.tm_q, bar(Gm::B_QFULL), 0, pc.u * N, 0, pc.b);
        }
        for (int t = pc.t0; t < pc.t1 && ok; t += T, ++n) {
          // the pages of this tile's boxes (one box of 64 tokens, or 2 of 32, or 4 of 16)
          int page[4], row0[4], nbox = 1;
          if (PAGED) {
            const int rows = 16 << rsh;
            nbox = (min(T, pc.t1 - t) + rows - 1) >> (4 + rsh);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (i < nbox) {
                const int tok = t + i * rows;
                const int col = p.page_shift >= 0 ? tok >> p.page_shift : tok / p.page_size;
                page[i] = load_dependent(p.page_table + (size_t)pc.b * p.max_pages + col);
                row0[i] = tok - col * p.page_size;
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (i < nbox && (unsigned)page[i] >= (unsigned)p.num_pages) {  // flag it, read page 0 instead
                atomicOr(&g_error_word, 4u);
                page[i] = 0;
              }
            }
          }
          const uint32_t col_bytes = PAGED ? (uint32_t)(nbox << (4 + rsh)) * 128u : (uint32_t)T * 128u;
          // columns [c, c + cols) of this tile to dst
          auto load = [&](const CUtensorMap* map, uint32_t dst, uint32_t full, int c, int cols) {
            mbar_arrive_expect_tx(full, col_bytes * cols);
            if (!PAGED) {
              tma_load_4d(dst, map, full, 0, t, c, pc.b);
            } else if (rsh == 2) {
              tma_load_4d(dst, map, full, 0, row0[0], c, page[0]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (i < nbox)
                  for (int k = 0; k < cols; ++k)
                    tma_load_4d(dst + (uint32_t)(k * T * 128 + (i << (4 + rsh)) * 128), map, full, 0, row0[i], c + k,
                                page[i]);
            }
          };
          if (second) {
            const int slot = n % Gm::NPE, fill = n / Gm::NPE;
            if (fill > 0 && !(ok = wait(Gm::B_PEEMPTY + slot, fill - 1))) break;
            load(&p.tm_pe, sbase + Gm::OFF_PE + slot * Gm::PE, bar(Gm::B_PEFULL + slot), 2 * NU, 1);
          }
          for (int k = second ? 1 : 0; k < NU; k += 2) {
            const int m = n * NU + k, slot = m % Gm::NUNIT, fill = m / Gm::NUNIT;
            if (fill > 0 && !(ok = wait(Gm::B_UEMPTY + slot, fill - 1))) break;
            load(&p.tm_unit, sbase + Gm::OFF_U + slot * Gm::UNIT, bar(Gm::B_UFULL + slot), 2 * k, 2);
          }
          if (!ok) break;
        }
        ++piece;
      }
      if (*abort_flag) {
        // copies in flight land before the CTA exits: the filled phases of every barrier this
        // warp armed (a phase that was never armed runs into the limit, which is harmless)
        const uint64_t t0 = globaltimer_ns();
        auto landed = [&](int b, int phase) {
          while (!mbar_try_wait(bar(b), (uint32_t)(phase & 1)) && globaltimer_ns() - t0 < p.timeout_ns) {
          }
        };
        const int last = n * NU + NU - 1;
        for (int m = last; m >= 0 && m > last - Gm::NUNIT; --m)
          if ((m % NU % 2 == 1) == second) landed(Gm::B_UFULL + m % Gm::NUNIT, m / Gm::NUNIT);
        if (second)
          for (int m = n; m >= 0 && m > n - Gm::NPE; --m) landed(Gm::B_PEFULL + m % Gm::NPE, m / Gm::NPE);
        else
          landed(Gm::B_QFULL, piece);
      }
    }
  } else if (warp == 1) {
    // ---- S^T of every tile
    constexpr uint32_t id_s = tc_idesc_bf16(64, N, false, false);
    bool ok = true, issued = false;
    while (ok && take(piece)) {
      ok = wait_all(Gm::B_QFULL, piece);
      for (int t = pc.t0; t < pc.t1 && ok; t += T, ++n) {
        const int sb = n & 1;
        // the softmax has read S of tile n - 2 (this slot's next phase needs tile n)
        if (n >= 2 && !(ok = wait_all(Gm::B_P + sb, (n >> 1) - 1))) break;
        const int valid = pc.t1 - t;  // tokens of this tile, if below T
        const uint32_t d = tmem + Gm::TCOL_S + sb * N;
        // the rotated part first: the last unit to land then has 8 products left
        const int slot_pe = n % Gm::NPE;
        if (!(ok = wait_all(Gm::B_PEFULL + slot_pe, n / Gm::NPE))) break;
        if (elect_one()) {
          tc_fence_after();
          const uint64_t da = tc_sdesc(sbase + Gm::OFF_PE + slot_pe * Gm::PE, 16, 1024, kTcSwizzle128B);
          const uint64_t db = tc_sdesc(sbase + Gm::OFF_Q + 2 * NU * N * 128, 16, 1024, kTcSwizzle128B);
#pragma unroll
          for (int i = 0; i < 4; ++i) tc_mma_ss(d, da + i * 2, db + i * 2, id_s, i > 0);
          tc_commit(bar(Gm::B_PEEMPTY + slot_pe));
        }
        issued = true;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < NU; ++k) {
          const int m = n * NU + k, slot = m % Gm::NUNIT;
          if (!(ok = wait_all(Gm::B_UFULL + slot, m / Gm::NUNIT))) break;
          const uint32_t unit = sbase + Gm::OFF_U + slot * Gm::UNIT;
          if (valid < T) {
            // rows past the sequence may hold anything, and 0 * NaN would poison O: zero them
            for (int e = valid * 8 + lane; e < T * 8; e += 32) {
              uint8_t* r = smem + Gm::OFF_U + slot * Gm::UNIT + swz<128>(e / 8, e % 8);
              *reinterpret_cast<uint4*>(r) = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4*>(r + T * 128) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (elect_one()) {
            tc_fence_after();
            const uint64_t da = tc_sdesc(unit, 16, 1024, kTcSwizzle128B);
            const uint64_t db = tc_sdesc(sbase + Gm::OFF_Q + 2 * k * N * 128, 16, 1024, kTcSwizzle128B);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              tc_mma_ss(d, da + (i / 4) * (T * 128 / 16) + (i % 4) * 2, db + (i / 4) * (N * 128 / 16) + (i % 4) * 2,
                        id_s, true);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) {
          tc_commit(bar(Gm::B_S + sb));
          if (t + T >= pc.t1) tc_commit(bar(Gm::B_QEMPTY));
        }
        __syncwarp();
      }
      ++piece;
    }
    if ((issued || !ok) && elect_one()) {  // everything issued completes before the tensor memory goes
      tc_commit(bar(Gm::B_FIN));
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(bar(Gm::B_FIN), 0) && globaltimer_ns() - t0 < p.timeout_ns) {
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---- O^T += C^T P^T of every tile
    constexpr uint32_t id_o = tc_idesc_bf16(128, N, true, false);
    bool ok = true, issued = false;
    while (ok && take(piece)) {
      // the epilogue has read the last piece's O
      if (piece > 0) ok = wait_all(Gm::B_OFREE, piece - 1);
      for (int t = pc.t0; t < pc.t1 && ok; t += T, ++n) {
        const int sb = n & 1;
        if (!(ok = wait_all(Gm::B_P + sb, n >> 1))) break;
        if (elect_one()) {
          tc_fence_after();
          const uint64_t db = tc_sdesc(sbase + Gm::OFF_P + (n % Gm::NP) * Gm::P_BYTES, 16, 1024, kTcSwizzle128B);
#pragma unroll
          for (int k = 0; k < NU; ++k) {
            const int slot = (n * NU + k) % Gm::NUNIT;
            const uint64_t da = tc_sdesc(sbase + Gm::OFF_U + slot * Gm::UNIT, T * 128, 1024, kTcSwizzle128B);
#pragma unroll
            for (int i = 0; i < T / 16; ++i)
              tc_mma_ss(tmem + k * N, da + i * (16 * 128 / 16), db + i * 2, id_o, t > pc.t0 || i > 0);
            tc_commit(bar(Gm::B_UEMPTY + slot));
          }
          tc_commit(bar(Gm::B_PV + sb));
        }
        issued = true;
        __syncwarp();
      }
      ++piece;
    }
    if (issued && elect_one()) {
      tc_commit(bar(Gm::B_FIN + 1));
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(bar(Gm::B_FIN + 1), 0) && globaltimer_ns() - t0 < p.timeout_ns) {
      }
    }
    __syncwarp();
  } else {
    // ---- softmax and epilogue: each warpgroup has NR rows (columns of S^T and O^T) of its
    // own, so its 128 threads meet on their own named barrier.  A wait that gives up only
    // marks the thread; the next vote takes the warpgroup out together.
    constexpr int NR = N / Gm::NWG;
    constexpr int NG = NR / 8;  // column groups of 8 rows
    const int w = warp & 3, wg = (warp >> 2) - 1, cb = wg * NR, mb = 1 + wg;
    const uint32_t lane_addr = (uint32_t)(32 * w) << 16;
    float* red = reinterpret_cast<float*>(smem + Gm::OFF_RED) + cb;
    float* colv = reinterpret_cast<float*>(smem + Gm::OFF_COL) + cb;
    float* colm = reinterpret_cast<float*>(smem + Gm::OFF_COLM) + cb;  // (a slow warp may still rescale by colv)
    const float kNegInf = -__int_as_float(0x7f800000);
    const int c2 = 2 * (lane & 3);  // this thread's rows: cb + 8 g + c2 and the next
    // where its stmatrix lane writes within P: row 8 (lane / 16) + lane % 8 of a pair of groups,
    // 16-byte chunk 2 w + (lane / 8) % 2 of tokens
    const int st_row = 8 * (lane >> 4) + (lane & 7);
    const uint32_t st_off = (uint32_t)(st_row * 128 + (((2 * w + ((lane >> 3) & 1)) ^ (st_row & 7)) << 4));
    bool ok = true;
    while (take(piece)) {
      const int L = max(0, min(p.seq_lens ? load_dependent(p.seq_lens + pc.b) : p.max_len, p.max_len));
      float m[2 * NG], l[2 * NG];
#pragma unroll
      for (int i = 0; i < 2 * NG; ++i) {
        m[i] = kNegInf;
        l[i] = 0.f;
      }
      bool stop = false;
      for (int t = pc.t0; t < pc.t1; t += T, ++n) {
        const int sb = n & 1;
        ok = wait(Gm::B_S + sb, n >> 1) && ok;
        ok = __all_sync(0xffffffffu, ok);
        float x[4 * NG];
        if (ok) {
          tc_fence_after();
          uint32_t r[4 * NG];
#pragma unroll
          for (int g = 0; g < NG; g += 2)
            tmem_ld_frag16(tmem + lane_addr + Gm::TCOL_S + sb * N + cb + 8 * g,
                           *reinterpret_cast<uint32_t(*)[8]>(r + 4 * g));
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 4 * NG; ++i) x[i] = __uint_as_float(r[i]) * p.scale_log2;
        } else {
#pragma unroll
          for (int i = 0; i < 4 * NG; ++i) x[i] = kNegInf;
        }
        // the first query token sees L - q_len + 1 tokens, each later one more
        if (t + T > L - p.q_len + 1) {
          const int tok = t + 16 * w + (lane >> 2);
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int lim = min(L, L - p.q_len + 1 + (pc.u * N + cb + 8 * g + c2 + e) / p.H);
              x[4 * g + e] = tok < lim ? x[4 * g + e] : kNegInf;
              x[4 * g + 2 + e] = tok + 8 < lim ? x[4 * g + 2 + e] : kNegInf;
            }
        }
        bool past = !ok;
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i)
          past |= fmaxf(x[4 * (i / 2) + i % 2], x[4 * (i / 2) + 2 + i % 2]) > m[i] + 24.f;
        if (named_bar_any(mb, 128, past)) {
          if (named_bar_any(mb, 128, !ok)) {
            stop = true;
            break;
          }
          // every row's maximum over the tile: over 8 lanes here, then over the warps
#pragma unroll
          for (int i = 0; i < 2 * NG; ++i) {
            float mx = fmaxf(x[4 * (i / 2) + i % 2], x[4 * (i / 2) + 2 + i % 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if (lane < 4) red[w * N + 8 * (i / 2) + c2 + i % 2] = mx;
          }
          named_bar_sync(mb, 128);
#pragma unroll
          for (int i = 0; i < 2 * NG; ++i) {
            const int c = 8 * (i / 2) + c2 + i % 2;
            const float mn = fmaxf(m[i], fmaxf(fmaxf(red[c], red[N + c]), fmaxf(red[2 * N + c], red[3 * N + c])));
            const float a = mn == kNegInf ? 1.f : exp2_approx(m[i] - mn);  // 0 while m is still -inf
            m[i] = mn;
            l[i] *= a;
            if (w == 0 && lane < 4) colv[c] = a;
          }
          named_bar_sync(mb, 128);
          if (t > pc.t0) {
            // O holds the tiles before this one, once the last of their products is done
            ok = wait(Gm::B_PV + ((n - 1) & 1), (n - 1) >> 1);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
              tc_fence_after();
#pragma unroll 1
              for (int e = 0; e < NU * NR; e += 16) {
                const int c0 = e % NR;
                const uint32_t at = tmem + lane_addr + (e / NR) * N + cb + c0;
                uint32_t o[16];
                tmem_ld16(at, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * colv[c0 + i]);
                tmem_st16(at, o);
              }
              tmem_st_wait();
            }
          }
        }
        // P^T of this tile; its buffer was last read by the product of tile n - NP
        if (n >= Gm::NP) {
          ok = wait(Gm::B_PV + ((n - Gm::NP) & 1), (n - Gm::NP) >> 1) && ok;
          ok = __all_sync(0xffffffffu, ok);
        }
#pragma unroll
        for (int g = 0; g < NG; g += 2) {
          uint32_t pk[4];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int i = 2 * (g + h);
              const float m0 = m[i] == kNegInf ? 0.f : m[i], m1 = m[i + 1] == kNegInf ? 0.f : m[i + 1];
              const uint32_t v = pack_bf16x2(exp2_approx(x[4 * (g + h) + 2 * half] - m0),
                                             exp2_approx(x[4 * (g + h) + 2 * half + 1] - m1));
              l[i] += bf16lo_to_f32(v);
              l[i + 1] += bf16hi_to_f32(v);
              pk[2 * h + half] = v;
            }
          stsm_x4_t(sbase + Gm::OFF_P + (n % Gm::NP) * Gm::P_BYTES + (cb / 8 + g) * 1024 + st_off, pk[0], pk[1], pk[2], pk[3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Gm::B_P + sb));
      }
      if (stop) break;
      // ---- the piece's sums: over 8 lanes, then over the warps in order
#pragma unroll
      for (int i = 0; i < 2 * NG; ++i) {
        float s = l[i];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        if (lane < 4) {
          const int c = 8 * (i / 2) + c2 + i % 2;
          red[w * N + c] = s;
          if (w == 0) colm[c] = m[i];
        }
      }
      ok = wait(Gm::B_PV + ((n - 1) & 1), (n - 1) >> 1) && ok;
      if (named_bar_any(mb, 128, !ok)) break;
      tc_fence_after();
      const int row0 = pc.u * N + cb;
      const int live = min(NR, p.rows - row0);  // rows of this warpgroup, if any
      const int slot = pc.slot;
      const bool whole = slot < 0;
      // (the meeting above made red and colm visible to all four warps)
      const int ctid = threadIdx.x & 127;
      float lsum = 0.f;
      if (ctid < NR) lsum = (red[ctid] + red[N + ctid]) + (red[2 * N + ctid] + red[3 * N + ctid]);
      if (!whole && ctid < live) p.part_ml[(size_t)slot * N + cb + ctid] = make_float2(colm[ctid], lsum);
      if (ctid < NR) colv[ctid] = whole ? (lsum > 0.f || lsum != lsum ? 1.f / lsum : 0.f) : 1.f;
      named_bar_sync(mb, 128);
#pragma unroll 1
      for (int k = 0; k < NU; ++k) {
#pragma unroll 1
        for (int c0 = 0; c0 < NR; c0 += 16) {
          if (c0 >= live) break;
          uint32_t o[16];
          tmem_ld16(tmem + lane_addr + k * N + cb + c0, o);
          tmem_ld_wait();
          const int d = k * 128 + 32 * w + lane;  // this lane's latent
          if (!whole) {
            float* dst = p.part_acc + ((size_t)slot * N + cb + c0) * R + d;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (c0 + i < live) dst[(size_t)i * R] = __uint_as_float(o[i]);
          } else {
            // two neighbouring lanes swap rows, so that each stores two latents of one row
            const int odd = lane & 1;
            __nv_bfloat16* dst = p.out + ((size_t)pc.b * p.rows + row0 + c0 + odd) * R + (d - odd);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float v0 = __uint_as_float(o[i]) * colv[c0 + i], v1 = __uint_as_float(o[i + 1]) * colv[c0 + i + 1];
              const float other = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
              const uint32_t word = odd ? pack_bf16x2(other, v1) : pack_bf16x2(v0, other);
              if (c0 + i + odd < live) *reinterpret_cast<uint32_t*>(dst + (size_t)i * R) = word;
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Gm::B_OFREE));
      ++piece;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Gm::TMEM_COLS);
  }
}

// Merge of the partials: for each row, M = max_j m_j over slots with l_j > 0, w_j =
// 2^(m_j - M), out = sum_j w_j acc_j / sum_j w_j l_j.  An item is 128 latents of a row, a
// float4 a lane.  Rows of up to 32 pieces are a warp's work, summed in ascending j.  A segment of more pieces fills more than 30 ranges, so there
// are few of them: warp 0 lists them in order, and each of their items takes a CTA, 16
// warps of slots (10 loads a thread in flight: 160 slots at once) whose sums are added in
// order.  Rows of empty sequences are zeroed.  All
// of the plan's work comes before the wait for the split kernel, whose CTAs let this one
// start only after their own wait: seq_lens is as they read it.
struct LatentCombineParams {
  const float* part_acc;
  const float2* part_ml;
  __nv_bfloat16* out;
  const int* seq_lens;
  int B, rows, U, N, ranges, max_len;
};

struct LatentCombineGeo {
  static constexpr int NTHREADS = 512, W = NTHREADS / 32, SHORT = 32;
  // shared: lane sums, weights of a long run, the list of long segments, the plan
  static constexpr int OFF_WTS = W * 32 * 16;
  __host__ __device__ static constexpr int off_list(int ranges) { return OFF_WTS + (ranges + 1 + 3) / 4 * 16; }
  __host__ __device__ static constexpr int off_plan(int ranges) { return off_list(ranges) + (ranges / (SHORT - 1) + 2 + 3) / 4 * 16; }
  static constexpr int smem_bytes(int ranges, int B) { return off_plan(ranges) + (2 * B + 2) * 4; }
};

template <int R>
__global__ void __launch_bounds__(512, 1) latent_combine_kernel(const LatentCombineParams p) {
  using Cg = LatentCombineGeo;
  extern __shared__ __align__(16) uint8_t csm[];
  float4* lane_sum = reinterpret_cast<float4*>(csm);               // [W][32]
  float* wts = reinterpret_cast<float*>(csm + Cg::OFF_WTS);        // [ranges], then the sum
  int* list = reinterpret_cast<int*>(csm + Cg::off_list(p.ranges));
  int* lens = reinterpret_cast<int*>(csm + Cg::off_plan(p.ranges));
  int* P = lens + p.B;
  constexpr int NCH = R / 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float kNegInf = -__int_as_float(0x7f800000);
  pdl_launch_dependents();
  build_plan_arrays(latent_length(p), p.B, p.max_len, kLatentGap, lens, P, 0, Cg::NTHREADS);
  const Plan pl = latent_plan(p.B, p.U, p.ranges, P);
  if (warp == 0) {
    int count = 0;
    const int nb_max = P[p.B + 1];
    if (nb_max > 0 && (nb_max - 1) / pl.q + 2 > Cg::SHORT) {
      for (int s0 = 0; s0 < p.B * p.U; s0 += 32) {
        const int seg = s0 + lane;
        const bool is_long = seg < p.B * p.U && segment_pieces(pl, lens, P, p.B, seg / p.U, seg % p.U) > Cg::SHORT;
        const unsigned m = __ballot_sync(0xffffffffu, is_long);
        if (is_long) list[1 + count + __popc(m & ((1u << lane) - 1))] = seg;
        count += __popc(m);
      }
    }
    if (lane == 0) list[0] = count;
  }
  __syncthreads();
  pdl_wait_primary();

  auto first_range = [&](int b, int u) { return (u * P[p.B] + P[b] + pl.gap) / pl.q; };
  auto acc_at = [&](int r0, int j, int col, int ch) {
    return reinterpret_cast<const float4*>(p.part_acc + ((size_t)latent_slot(r0, j) * p.N + col) * R + ch * 128) + lane;
  };
  auto ml_at = [&](int r0, int j, int col) { return __ldcg(p.part_ml + (size_t)latent_slot(r0, j) * p.N + col); };
  auto is_live = [](float l) { return l > 0.f || l != l; };
  auto put = [&](int b, int row, int ch, float4 s, float den) {
    const float inv = is_live(den) ? 1.f / den : 0.f;
    uint2 o;
    o.x = pack_bf16x2(s.x * inv, s.y * inv);
    o.y = pack_bf16x2(s.z * inv, s.w * inv);
    reinterpret_cast<uint2*>(p.out + ((size_t)b * p.rows + row) * R + ch * 128)[lane] = o;
  };
  // ---- long segments
  const int nlong = list[0], per_seg = p.N * NCH;
  for (int item = blockIdx.x; item < nlong * per_seg; item += gridDim.x) {
    const int seg = list[1 + item / per_seg], in_seg = item % per_seg;
    const int b = seg / p.U, u = seg % p.U, col = in_seg / NCH, ch = in_seg % NCH;
    const int row = u * p.N + col;
    if (row >= p.rows) continue;
    const int n = segment_pieces(pl, lens, P, p.B, b, u), r0 = first_range(b, u);
    constexpr int KB = 10;
    float4 a[KB];
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const int j = warp + Cg::W * k;
      a[k] = j < n ? __ldcg(acc_at(r0, j, col, ch)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (warp == 0) {  // the weights, while the loads are in flight
      constexpr int KM = 5;  // 160 slots at a time
      float2 v[KM];
      float M = kNegInf;
      for (int j0 = 0; j0 < n; j0 += 32 * KM) {
#pragma unroll
        for (int k = 0; k < KM; ++k) {
          const int j = j0 + lane + 32 * k;
          v[k] = j < n ? ml_at(r0, j, col) : make_float2(kNegInf, 0.f);
        }
#pragma unroll
        for (int k = 0; k < KM; ++k)
          if (is_live(v[k].y)) M = fmaxf(M, v[k].x);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      float den = 0.f;
      for (int j0 = 0; j0 < n; j0 += 32 * KM) {
#pragma unroll
        for (int k = 0; k < KM; ++k) {
          const int j = j0 + lane + 32 * k;
          if (n > 32 * KM) v[k] = j < n ? ml_at(r0, j, col) : make_float2(kNegInf, 0.f);
          const float wj = is_live(v[k].y) ? exp2_approx(v[k].x - M) : 0.f;
          if (j < n) wts[j] = wj;
          if (wj != 0.f) den += wj * v[k].y;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
      if (lane == 0) wts[p.ranges] = den;
    }
    __syncthreads();
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = warp; j0 < n; j0 += KB * Cg::W) {
      if (j0 != warp) {
#pragma unroll
        for (int k = 0; k < KB; ++k) {
          const int j = j0 + Cg::W * k;
          a[k] = j < n ? __ldcg(acc_at(r0, j, col, ch)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        const int j = j0 + Cg::W * k;
        const float wj = j < n ? wts[j] : 0.f;
        if (wj != 0.f) {
          s.x += wj * a[k].x;
          s.y += wj * a[k].y;
          s.z += wj * a[k].z;
          s.w += wj * a[k].w;
        }
      }
    }
    lane_sum[warp * 32 + lane] = s;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int k = 1; k < Cg::W; ++k) {
        const float4 v = lane_sum[k * 32 + lane];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      put(b, row, ch, s, wts[p.ranges]);
    }
    __syncthreads();
  }
  // ---- short segments and empty sequences: CPI chunks of a row are a warp's work, 16 loads a
  // lane in flight.  Whole rows when there are about enough for every warp, else chunks: a
  // row's fixed work (divisions, shuffles) is an item's (2048 rows on 2432 warps, 5 pieces
  // each: the call 42.1 us with whole rows, 45.9 with chunks).  Neighbouring rows, which have
  // the same number of pieces, go to different CTAs: with them in one, a long sequence's few CTAs
  // did most of the work (64 sequences of 1 to 32768 tokens: 66.6 us, now 61.6).
  auto merge_short = [&](auto cpi) {
    constexpr int CPI = decltype(cpi)::value, PARTS = NCH / CPI, KB = 16 / CPI;
    const unsigned items = (unsigned)p.B * p.rows * PARTS;
    for (unsigned item = blockIdx.x + gridDim.x * warp; item < items; item += gridDim.x * Cg::W) {
      const int ch = item % PARTS * CPI, grow = item / PARTS;
      const int b = grow / p.rows, row = grow - b * p.rows;
      const int u = row / p.N, col = row - u * p.N;
      const int n = segment_pieces(pl, lens, P, p.B, b, u);
      if (n == 1 || n > Cg::SHORT) continue;
      const int r0 = n > 0 ? first_range(b, u) : 0;
      float4 a[KB][CPI];
      auto fetch = [&](int j0) {
#pragma unroll
        for (int j = 0; j < KB; ++j)
#pragma unroll
          for (int c = 0; c < CPI; ++c)
            a[j][c] = j0 + j < n ? __ldcg(acc_at(r0, j0 + j, col, ch + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
      };
      fetch(0);
      const float2 ml = lane < n ? ml_at(r0, lane, col) : make_float2(kNegInf, 0.f);
      const bool live = is_live(ml.y);
      float M = live ? ml.x : kNegInf;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float wgt = live ? exp2_approx(ml.x - M) : 0.f;
      float den = 0.f;
      float4 s[CPI];
#pragma unroll
      for (int c = 0; c < CPI; ++c) s[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int j0 = 0; j0 < n; j0 += KB) {
        if (j0 > 0) fetch(j0);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          const float wj = __shfl_sync(0xffffffffu, wgt, (j0 + j) & 31), lj = __shfl_sync(0xffffffffu, ml.y, (j0 + j) & 31);
          if (j0 + j < n && wj != 0.f) {
            den += wj * lj;
#pragma unroll
            for (int c = 0; c < CPI; ++c) {
              s[c].x += wj * a[j][c].x;
              s[c].y += wj * a[j][c].y;
              s[c].z += wj * a[j][c].z;
              s[c].w += wj * a[j][c].w;
            }
          }
        }
      }
#pragma unroll
      for (int c = 0; c < CPI; ++c) put(b, row, ch + c, s[c], den);
    }
  };
  if ((unsigned)p.B * p.rows * 4 >= gridDim.x * Cg::W * 3)
    merge_short(std::integral_constant<int, NCH>{});
  else
    merge_short(std::integral_constant<int, 1>{});
}

}  // namespace da
