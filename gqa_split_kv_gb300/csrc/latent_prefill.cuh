// Causal prefill over keys and values expanded from latent vectors (the expanded form
// of latent attention), on the 5th-generation tensor cores.
//
// Head h's key at token t is [k_nope[t, h], k_rope[t]]: D elements of its own and 64
// rotated ones that all heads share, read from one place.  Values have D elements.
//   S = q[0:D] k_nope^T + q[D:D+64] k_rope^T,  O = softmax(scale S) v
// Operations 2 (2 D + 64) a (row, visible key), bytes of K and V once a query block: a
// dense contraction, bound by the tensor cores and, beside them, by one exponential a
// (row, key): with 320 products a weight at D = 128 the two take about the same time.
//
// The engine is prefill_tc.cuh's with two query tiles: a CTA owns 256 query tokens of one
// head, tile A and tile B of 128 rows (tensor memory lanes); S_A, S_B (128 columns), O_A,
// O_B (D) fill tensor memory; each tile has a softmax warpgroup, one thread a row, and
// while one works the tensor cores run the other's products:
//   P_A V_j, S_A = Q_A K_{j+1}^T, P_B V_j, S_B = Q_B K_{j+1}^T.
// What differs is the shared memory.  The queries take 96 KB at D = 128, so K and V come
// through one ring of 16 KB granules, each freed by its own last product: K_j is D / 64 + 1
// granules of 128 keys x 64 elements (the last one the shared part), V_j granules of 64
// keys x 128 elements (D = 128) or 128 x 64.  Five a tile at D = 128 and eight in the ring:
// P_B V_j frees two that K_{j+2} takes, 1290 cycles of products before it is used.  A ring
// of whole tiles would hold one and a half of 128 keys, and tiles of 64 keys take 48
// instead of 32 cycles an MMA.
//
// A few query blocks (a chunk after a long prefix, few heads) leave most SMs idle.  Then a
// block's key tiles are cut into up to `parts` equal parts (prefill_cut.cuh), each a CTA's,
// which leaves (O, m, l) unnormalised in fp32; latent_prefill_merge joins them.  A block of one
// part is written at once.
//
// More blocks than SMs: a CTA that has issued its last loads asks for the index of one that
// has not started (clusterlaunchcontrol) and goes on with it, so the next block's queries and
// keys load and its first scores are taken while the last one's output is written.  The launch order,
// longest blocks first, and so the balance, stay the hardware's: 4096-token prompt, 32 heads,
// D = 128: 131.5 us, 144.8 with a CTA a block.
//
// Registers: the issuing warps need 120; with 72 the spills between MMAs cost 8% (141.9
// us), and the softmax warps need no more than 192.
//
// Bound by the tensor cores at the clock that the card holds under them (1.5 GHz), where a
// tile of both query tiles takes 1.9 us, 1.7 of them its 40 MMAs: the prompt above is 131.5 us,
// the operations under the mask 87.3 at the measured peak; the rest is the clock, the masked
// halves of diagonal tiles (3%) and the start and end.  4 sequences of 500 new tokens up to 3000, 16 heads:
// 48.2 us, floor 13.6: 128 query blocks on 152 SMs, and the longest is the call's time.
// Tried and dropped there: all blocks on one line, cut into equal ranges (46.8 us; the merge of 37 MB
// of pieces takes most of what the balance gives, and a prompt takes 151).
#pragma once

#include <cstdint>

#include "device_error.cuh"
#include "prefill_cut.cuh"
#include "ptx.cuh"
#include "tc05.cuh"

namespace da {

struct LatentPrefillParams {
  CUtensorMap tm_q;   // [B][H][W / 64][q_len][64], boxes of 128 tokens and every column
  CUtensorMap tm_k;   // [B][H][D / 64][tokens][64], boxes of 128 tokens and one column
  CUtensorMap tm_v;   // the same, boxes of VKEYS tokens and every column
  CUtensorMap tm_pe;  // [B][tokens][64], boxes of 128 tokens
  __nv_bfloat16* out;      // [B, q_len, H, D]
  const int* seq_lens;     // [B] or null (every sequence max_len tokens)
  float* part_acc;         // [unit][part][D][256]: parts' O (with more than one part)
  float2* part_ml;         // [unit][part][256], m in log2 units
  int parts;               // CTAs a unit: parts that its keys may have
  int more;                // not every CTA runs at once: CTAs take over others' indices
  int B, q_len, H, nqb;
  int grp;                 // (sequence, head) units per launch group (their K/V fit in L2 together)
  int grp_by_length;       // that is by the capacity: the kernel takes the longest sequence's tokens
  int max_len;
  float scale_log2;
  unsigned long long timeout_ns;
};

template <int D>
struct LatentPrefillGeo {
  static constexpr int M = 128, BK = 128, NQT = 2;  // rows a query tile, keys a tile
  static constexpr int BQ = NQT * M;                // query tokens a CTA
  static constexpr int W = D + 64;                  // elements of a query
  static constexpr int NKG = W / 64;                // K granules a tile
  static constexpr int G = 16384;                   // bytes a granule
  static constexpr int VKEYS = G / (2 * D);         // keys of a V granule
  static constexpr int NVG = BK / VKEYS;
  static constexpr int PER = NKG + NVG;             // granules a tile
  static constexpr int QT_BYTES = M * W * 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_G = NQT * QT_BYTES;
  static constexpr int NG_FIT = (227 * 1024 - 1024 - 1024 - OFF_G) / G;
  static constexpr int NG = NG_FIT < 12 ? NG_FIT : 12;
  static constexpr int OFF_BAR = OFF_G + NG * G;
  static constexpr int BAR_FULL = 0, BAR_EMPTY = NG, BAR_S = 2 * NG, BAR_P = BAR_S + 2, BAR_O = BAR_P + 2,
                       BAR_Q = BAR_O + 2, BAR_QE = BAR_Q + 2, BAR_NEXT = BAR_QE + 2, BAR_READ = BAR_NEXT + 2, BAR_ANSWER = BAR_READ + 2,
                       BAR_FIN = BAR_ANSWER + 1, NBAR = BAR_FIN + 1;
  static constexpr int OFF_ANSWER = OFF_BAR + (NBAR + 1) / 2 * 16;  // to the request for a next index
  static constexpr int OFF_PIECE = OFF_ANSWER + 16;                 // this piece and the next
  static constexpr int OFF_MISC = OFF_PIECE + 2 * 48;               // tensor memory base, abort flag, grp
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static constexpr int TCOL_O = 2 * BK;             // S of tile t at t BK, O at TCOL_O + t D
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int NTHREADS = 128 + 128 * NQT;
  // registers after the split: producers and MMA issue, softmax
  static constexpr int REG_LOW = 120, REG_HIGH = 192;
  static constexpr int REG_POOL_NEEDED = 128 * REG_LOW + 128 * NQT * REG_HIGH;
  static_assert(NG >= PER + NVG && SMEM <= 227 * 1024, "the ring holds a tile's K and two of V");
  static_assert(TCOL_O + NQT * D <= 512, "tensor memory");
};

template <int N>
__device__ __forceinline__ void latent_setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void latent_setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// A CTA's work of one index: tiles [j0, j0 + n) of query block qb of (b, h).  Groups of grp
// (b, h) units, latest query blocks (the longest) first; a unit's parts together.
struct PrefillPiece {
  int b, h, qb;
  int L, nq, base, kv_end;  // length, rows, position of query token 0, keys some row sees
  int j0, n, n_a;           // n_a: of the n tiles, those that query tile A's rows see some of
  int slot;                 // of the part; -1: the whole block
  int any;                  // 0: no part of this index; -1: no more pieces
  __device__ __forceinline__ void set(const LatentPrefillParams& p, int grp, int index) volatile {
    constexpr int BQ = 256, BK = 128;
    if (index < 0) {
      any = -1;
      return;
    }
    const int part = index % p.parts, unit = index / p.parts;
    const int nbh = p.B * p.H;
    const long long per_grp = (long long)p.nqb * grp;
    const int gi = (int)(unit / per_grp);
    const int gsz = min(grp, nbh - gi * grp);
    const int in_g = (int)(unit - gi * per_grp);
    const int bh = gi * grp + in_g % gsz;
    const int qb_ = p.nqb - 1 - in_g / gsz, b_ = bh / p.H;
    int len = p.seq_lens ? load_dependent(p.seq_lens + b_) : p.max_len;
    len = len < 0 ? 0 : (len > p.max_len ? p.max_len : len);
    const int rows = min(BQ, p.q_len - qb_ * BQ), first = len - p.q_len;
    const int end = max(0, min(len, first + qb_ * BQ + rows)), tiles = (end + BK - 1) / BK;
    const int nparts = prefill_block_parts(tiles, p.parts);
    const int from = part < nparts ? prefill_part_begin(tiles, part, nparts) : 0;
    const int count = part < nparts ? prefill_part_begin(tiles, part + 1, nparts) - from : 0;
    const int end_a = max(0, min(len, first + qb_ * BQ + min(rows, BQ / 2)));
    b = b_;
    h = bh - b_ * p.H;
    qb = qb_;
    L = len;
    nq = rows;
    base = first;
    kv_end = end;
    j0 = from;
    n = count;
    n_a = max(0, min(count, (end_a + BK - 1) / BK - from));
    slot = nparts == 1 ? -1 : (bh * p.nqb + qb_) * p.parts + part;
    any = part < nparts;
  }
};

// A CTA that has finished its own index goes on with one that has not started: it asks the
// launch hardware to cancel a waiting CTA and takes that one's index.
__device__ __forceinline__ void request_next(uint32_t answer, uint32_t mbar) {
  mbar_arrive_expect_tx(mbar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   answer),
               "r"(mbar)
               : "memory");
}
// The index of the cancelled CTA (a grid of one dimension), or -1: none was waiting.
__device__ __forceinline__ int next_index(uint32_t answer) {
  int x;
  asm volatile(
      "{\n\t"
      ".reg .b128 a;\n\t"
      ".reg .pred p;\n\t"
      "ld.shared.b128 a, [%1];\n\t"
      "mov.b32 %0, -1;\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, a;\n\t"
      "}"
      : "=r"(x)
      : "r"(answer)
      : "memory");
  return x;
}

template <int D>
__global__ void __launch_bounds__(LatentPrefillGeo<D>::NTHREADS, 1)
    latent_prefill_kernel(const __grid_constant__ LatentPrefillParams p) {
  using Gm = LatentPrefillGeo<D>;
  constexpr int BK = Gm::BK, M = Gm::M;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  auto bar = [&](int i) -> uint32_t { return sbase + Gm::OFF_BAR + 8 * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Gm::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float kNegInf = -__int_as_float(0x7f800000);

  pdl_wait_primary();  // (what precedes this call in the stream)
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < Gm::NG; ++i) {
      mbar_init(bar(Gm::BAR_FULL + i), 1);
      mbar_init(bar(Gm::BAR_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(Gm::BAR_S + i), 1);
      mbar_init(bar(Gm::BAR_P + i), 4);  // one arrival a warp
      mbar_init(bar(Gm::BAR_O + i), 1);
      mbar_init(bar(Gm::BAR_Q + i), 1);
      mbar_init(bar(Gm::BAR_QE + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(Gm::BAR_NEXT + i), 1);
      mbar_init(bar(Gm::BAR_READ + i), 1 + 4 * Gm::NQT);  // the issuing warp's and the softmax warps'
    }
    mbar_init(bar(Gm::BAR_ANSWER), 1);
    mbar_init(bar(Gm::BAR_FIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&p.tm_q);
    prefetch_tensormap(&p.tm_k);
    prefetch_tensormap(&p.tm_v);
    prefetch_tensormap(&p.tm_pe);
  }
  if (warp == 1) {
    tmem_alloc(sbase + Gm::OFF_MISC, Gm::TMEM_COLS);
    tmem_relinquish();
  }
  int grp = p.grp;
  if (p.grp_by_length && warp == 2) {
    int longest = 0;
    for (int b = lane; b < p.B; b += 32) longest = max(longest, load_dependent(p.seq_lens + b));
    grp = prefill_group(min(__reduce_max_sync(0xffffffffu, longest), p.max_len), D, (long long)p.B * p.H);
  }
  if (threadIdx.x == 64) {
    reinterpret_cast<volatile PrefillPiece*>(smem + Gm::OFF_PIECE)->set(p, grp, blockIdx.x);
    *reinterpret_cast<int*>(smem + Gm::OFF_MISC + 8) = grp;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Gm::OFF_MISC);
  auto wait = [&](int i, int phase) { return wait_bounded(bar(i), (uint32_t)(phase & 1), abort_flag, p.timeout_ns); };
  // The pieces a CTA works through: its own index's, then those of the indices it takes over.
  // Piece k lies in buffer k & 1; the producer writes piece k + 1 there when every role has
  // left piece k - 1.
  volatile PrefillPiece* pieces = reinterpret_cast<volatile PrefillPiece*>(smem + Gm::OFF_PIECE);
  auto leave = [&](int k) {  // whole warps: piece k is done; true when there is another
    __syncwarp();
    if (!p.more) return false;
    if (lane == 0) mbar_arrive(bar(Gm::BAR_READ + (k & 1)));
    return __all_sync(0xffffffffu, wait(Gm::BAR_NEXT + ((k + 1) & 1), k >> 1)) && pieces[(k + 1) & 1].any >= 0;
  };
  // granule g of the CTA's tile j (counted over its pieces): K columns 0 .. NKG - 1, then V
  auto slot_of = [&](int j, int g) { return (j * Gm::PER + g) % Gm::NG; };
  auto fill_of = [&](int j, int g) { return (j * Gm::PER + g) / Gm::NG; };
  auto addr_of = [&](int j, int g) { return sbase + Gm::OFF_G + (uint32_t)(slot_of(j, g) * Gm::G); };

  if (warp < 4) {
    // ---- first warpgroup: every warp gives registers up at the same instruction
    latent_setmaxnreg_dec<Gm::REG_LOW>();
    if (warp == 0) {
      // ---- producer: granules in the order the products use them.  The wait for the free of
      // granule m - NG is by its slot's phase, whose next one needs granule m.
      if (lane == 0) {
        bool ok = true;
        int last = -1, tiles = 0, fills[2] = {0, 0};  // of the pieces before
        bool waiting = false;  // for a request's answer
        int k = 0;
        do {
          volatile PrefillPiece& pc = pieces[k & 1];
          const int b = pc.b, h = pc.h, n = pc.n, nqt = pc.nq > M ? 2 : 1, q0 = pc.qb * Gm::BQ, j0 = pc.j0;
          // query tiles, [W / 64][M][64] each; zeros past q_len
          for (int t = 0; t < nqt && n > 0; ++t) {
            if (fills[t] > 0 && !(ok = wait(Gm::BAR_QE + t, fills[t] - 1))) break;
            ++fills[t];
            mbar_arrive_expect_tx(bar(Gm::BAR_Q + t), Gm::QT_BYTES);
            tma_load_5d(sbase + Gm::OFF_Q + t * Gm::QT_BYTES, &p.tm_q, bar(Gm::BAR_Q + t), 0, q0 + t * M, 0, h, b);
          }
          for (int j = 0; j < n && ok; ++j) {
            const int t = (j0 + j) * BK;
#pragma unroll 1
            for (int g = 0; g < Gm::PER; ++g) {
              const int fill = fill_of(tiles + j, g), slot = slot_of(tiles + j, g);
              if (fill > 0 && !(ok = wait(Gm::BAR_EMPTY + slot, fill - 1))) break;
              const uint32_t full = bar(Gm::BAR_FULL + slot);
              mbar_arrive_expect_tx(full, Gm::G);
              if (g < Gm::NKG - 1)
                tma_load_5d(addr_of(tiles + j, g), &p.tm_k, full, 0, t, g, h, b);
              else if (g == Gm::NKG - 1)
                tma_load_3d(addr_of(tiles + j, g), &p.tm_pe, full, 0, t, b);
              else
                tma_load_5d(addr_of(tiles + j, g), &p.tm_v, full, 0, t + (g - Gm::NKG) * Gm::VKEYS, 0, h, b);
              last = (tiles + j) * Gm::PER + g;
            }
          }
          tiles += n;
          if (!ok || !p.more) break;
          // asked only now, with this piece's loads issued: a CTA that asks at its start takes
          // over indices whose SM is about to be free
          const uint32_t answer = sbase + Gm::OFF_ANSWER;
          request_next(answer, bar(Gm::BAR_ANSWER));
          waiting = true;
          if (!(ok = wait(Gm::BAR_ANSWER, k))) break;
          waiting = false;
          if (k > 0 && !(ok = wait(Gm::BAR_READ + ((k + 1) & 1), (k - 1) >> 1))) break;
          ++k;
          pieces[k & 1].set(p, *reinterpret_cast<volatile int*>(smem + Gm::OFF_MISC + 8), next_index(answer));
          fence_proxy_async_smem();  // the answer is read before another is asked for
          mbar_arrive(bar(Gm::BAR_NEXT + (k & 1)));
        } while (pieces[k & 1].any >= 0);
        if (*abort_flag) {  // copies in flight land before the CTA exits
          const uint64_t t0 = globaltimer_ns();
          while (waiting && !mbar_try_wait(bar(Gm::BAR_ANSWER), (uint32_t)(k & 1)) &&
                 globaltimer_ns() - t0 < p.timeout_ns) {
          }
          for (int t = 0; t < 2; ++t)
            while (fills[t] > 0 && !mbar_try_wait(bar(Gm::BAR_Q + t), (uint32_t)((fills[t] - 1) & 1)) &&
                   globaltimer_ns() - t0 < p.timeout_ns) {
            }
          for (int m = last; m >= 0 && m > last - Gm::NG; --m)
            while (!mbar_try_wait(bar(Gm::BAR_FULL + m % Gm::NG), (uint32_t)((m / Gm::NG) & 1)) &&
                   globaltimer_ns() - t0 < p.timeout_ns) {
            }
        }
      }
    } else if (warp == 1) {
      // ---- MMA issue (one lane); the warp zeroes V rows past the keys of the last tile
      constexpr uint32_t id_s = tc_idesc_bf16(M, BK, false, false);
      constexpr uint32_t id_o = tc_idesc_bf16(M, D, false, true);
      int nqt = 1, tiles = 0, kv_end = 0, j0 = 0;  // query tiles with rows; tiles of the pieces before
      auto wait_all = [&](int i, int phase) { return __all_sync(0xffffffffu, wait(i, phase)) != 0; };
      // granules [g0, g1) of tile j have landed (query tile A waits for both)
      auto landed = [&](int j, int g0, int g1) {
        bool there = true;
        for (int g = g0; g < g1; ++g) there = wait(Gm::BAR_FULL + slot_of(tiles + j, g), fill_of(tiles + j, g)) && there;
        return __all_sync(0xffffffffu, there) != 0;
      };
      // one thread: S_t = Q_t K_j^T; the granules are freed after the last query tile, the
      // queries after the piece's last tile
      auto issue_qk = [&](int t, int j, bool last) {
#pragma unroll
        for (int g = 0; g < Gm::NKG; ++g) {
          const uint64_t da = tc_sdesc(sbase + Gm::OFF_Q + t * Gm::QT_BYTES + g * (M * 128), 16, 1024, kTcSwizzle128B);
          const uint64_t db = tc_sdesc(addr_of(tiles + j, g), 16, 1024, kTcSwizzle128B);
#pragma unroll
          for (int i = 0; i < 4; ++i) tc_mma_ss(tmem + t * BK, da + 2 * i, db + 2 * i, id_s, g > 0 || i > 0);
          if (t == nqt - 1) tc_commit(bar(Gm::BAR_EMPTY + slot_of(tiles + j, g)));
        }
        tc_commit(bar(Gm::BAR_S + t));
        if (last) tc_commit(bar(Gm::BAR_QE + t));
      };
      // one thread: O_t += P_t V_j with P_t from the S buffer
      auto issue_pv = [&](int t, int j) {
#pragma unroll
        for (int g = 0; g < Gm::NVG; ++g) {
          const uint64_t db = tc_sdesc(addr_of(tiles + j, Gm::NKG + g), Gm::VKEYS * 128, 1024, kTcSwizzle128B);
#pragma unroll
          for (int i = 0; i < Gm::VKEYS / 16; ++i)
            tc_mma_ts(tmem + Gm::TCOL_O + t * D, tmem + t * BK + 8 * (g * (Gm::VKEYS / 16) + i), db + i * 128, id_o,
                      j > 0 || g > 0 || i > 0);
          if (t == nqt - 1) tc_commit(bar(Gm::BAR_EMPTY + slot_of(tiles + j, Gm::NKG + g)));
        }
      };
      // V rows at or past kv_end may hold anything (0 * NaN would poison O): zero them
      auto zero_tail = [&](int j) {
        for (int g = 0; g < Gm::NVG; ++g) {
          const int r0 = max(0, kv_end - ((j0 + j) * BK + g * Gm::VKEYS));
          uint8_t* vs = smem + Gm::OFF_G + slot_of(tiles + j, Gm::NKG + g) * Gm::G;
          for (int e = r0 * 8 + lane; e < Gm::VKEYS * 8; e += 32)
            for (int c = 0; c < D / 64; ++c)
              *reinterpret_cast<uint4*>(vs + c * (Gm::VKEYS * 128) + swz<128>(e / 8, e % 8)) =
                  make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
      };
      bool ok = true;
      int fills[2] = {0, 0}, done[2] = {0, 0};  // pieces and key tiles of each query tile so far
      int k = 0;
      do {
        volatile PrefillPiece& pc = pieces[k & 1];
        if (pc.n == 0) continue;
        const int ntiles = pc.n, ntiles_a = pc.n_a;
        nqt = pc.nq > M ? 2 : 1;
        kv_end = pc.kv_end;
        j0 = pc.j0;
        ok = wait_all(Gm::BAR_Q, fills[0]++) && landed(0, 0, Gm::NKG);
        if (!ok) break;
        if (elect_one()) {
          tc_fence_after();
          if (ntiles_a > 0)
            issue_qk(0, 0, ntiles_a == 1);
          else
            tc_commit(bar(Gm::BAR_QE));
        }
        __syncwarp();
        if (nqt == 2) {
          if (!(ok = wait_all(Gm::BAR_Q + 1, fills[1]++))) break;
          if (elect_one()) {
            tc_fence_after();
            issue_qk(1, 0, ntiles == 1);
          }
          __syncwarp();
        }
        for (int j = 0; j < ntiles && ok; ++j) {
          const bool more = j + 1 < ntiles;
          // A: P_A V_j, then S_A of tile j + 1 once its keys are there
          ok = landed(j, Gm::NKG, Gm::PER);
          if (!ok) break;
          if ((j0 + j + 1) * BK > kv_end) zero_tail(j);
          if (j < ntiles_a) {
            if (!(ok = wait_all(Gm::BAR_P, done[0]++))) break;
            if (elect_one()) {
              tc_fence_after();
              issue_pv(0, j);
              if (j + 1 == ntiles_a) tc_commit(bar(Gm::BAR_O));
            }
            __syncwarp();
          }
          if (more) {
            if (!(ok = landed(j + 1, 0, Gm::NKG))) break;
            if (j + 1 < ntiles_a && elect_one()) {
              tc_fence_after();
              issue_qk(0, j + 1, j + 2 == ntiles_a);
            }
            __syncwarp();
          }
          if (nqt == 2) {  // B: the same tiles
            if (!(ok = wait_all(Gm::BAR_P + 1, done[1]++))) break;
            if (elect_one()) {
              tc_fence_after();
              issue_pv(1, j);
              if (more)
                issue_qk(1, j + 1, j + 2 == ntiles);
              else
                tc_commit(bar(Gm::BAR_O + 1));
            }
            __syncwarp();
          }
        }
        tiles += ntiles;
      } while (ok && leave(k++));
      // before the tensor memory is freed, every MMA issued must have completed
      if (fills[0] > 0 && elect_one()) {
        tc_commit(bar(Gm::BAR_FIN));
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(bar(Gm::BAR_FIN), 0) && globaltimer_ns() - t0 < p.timeout_ns) {
        }
      }
      __syncwarp();
    }  // warps 2 and 3: idle
  } else {
    // ---- softmax and epilogue of query tile qt: one thread per row (tensor memory lane)
    latent_setmaxnreg_inc<Gm::REG_HIGH>();
    const int qt = (warp >> 2) - 1;
    const int row = lane + 32 * (warp & 3);
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_addr = tmem + lane_addr + Gm::TCOL_O + qt * D;
    const uint32_t s_addr = tmem + lane_addr + qt * BK;
    const int tok = qt * M + row;               // this row's token within the block
    const bool fold = p.scale_log2 > 0.f;  // a positive scale goes into the exponent's fma
    const float sc = fold ? p.scale_log2 : 1.f;
    bool ok = true;
    int done = 0, ends = 0;  // key tiles, and pieces that had some, so far
    int k = 0;
    do {
      volatile PrefillPiece& pc = pieces[k & 1];
      if (!pc.any || (qt > 0 && pc.nq <= M)) continue;  // no rows
      const int j0 = pc.j0, q0 = pc.qb * Gm::BQ;
      const int nt = qt == 0 ? pc.n_a : pc.n;           // this query tile's key tiles
      const int lim = tok < pc.nq ? max(0, min(pc.L, pc.base + q0 + tok + 1)) : 0;  // keys this row sees
      const int lim_first = max(0, min(pc.L, pc.base + q0 + qt * M + 1));       // keys every row of the tile sees
      float m = kNegInf, l = 0.f;
      for (int j = 0; j < nt; ++j) {
        ok = __all_sync(0xffffffffu, wait(Gm::BAR_S + qt, done++));
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
          const int left = lim - (j0 + j) * BK;  // keys of this tile that the row sees
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
        // yet, or whose weights sum past 2^14, takes its maximum and raises m to it.  The
        // stores in weights() are the whole warp's, so every call is warp-uniform.
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
        const float alpha = raise ? exp2_approx(m - m_new) : 1.f;  // 0 while m is still -inf
        if (__any_sync(0xffffffffu, raise && m != kNegInf) && j > 0) {
          // S of tile j was issued after P V of tile j - 1 by the same thread, and its commit
          // covers every MMA before it: O is complete
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
        if (lane == 0) mbar_arrive(bar(Gm::BAR_P + qt));
      }
      // ---- normalise and write the tile's rows (a row that saw nothing: zeros)
      if (ok && nt > 0) ok = __all_sync(0xffffffffu, wait(Gm::BAR_O + qt, ends++));
      if (ok) {
        tc_fence_after();
        const bool has_row = tok < pc.nq, whole = pc.slot < 0;
        if (!whole) {
          // the part as it is, [D][256]: 32 lanes store 32 rows of a column
          const size_t slot = (size_t)pc.slot;
          float* acc = p.part_acc + slot * D * Gm::BQ + tok;
#pragma unroll 1
          for (int c0 = 0; c0 < D && nt > 0; c0 += 32) {  // (l is 0 with no tile, and nothing else read)
            uint32_t r[32];
            tmem_ld32(o_addr + c0, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[(size_t)(c0 + i) * Gm::BQ] = __uint_as_float(r[i]);
          }
          p.part_ml[slot * Gm::BQ + tok] = make_float2(m, l);
        }
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
        __nv_bfloat16* dst = p.out + (((size_t)pc.b * p.q_len + pc.qb * Gm::BQ + tok) * p.H + pc.h) * D;
#pragma unroll 1
        for (int c0 = 0; c0 < D && whole; c0 += 32) {
          uint32_t r[32];
          if (nt > 0) {
            tmem_ld32(o_addr + c0, r);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = 0u;
          }
          if (has_row) {
            uint4* o = reinterpret_cast<uint4*>(dst + c0);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              o[k] = make_uint4(pack_bf16x2(__uint_as_float(r[8 * k + 0]) * inv, __uint_as_float(r[8 * k + 1]) * inv),
                                pack_bf16x2(__uint_as_float(r[8 * k + 2]) * inv, __uint_as_float(r[8 * k + 3]) * inv),
                                pack_bf16x2(__uint_as_float(r[8 * k + 4]) * inv, __uint_as_float(r[8 * k + 5]) * inv),
                                pack_bf16x2(__uint_as_float(r[8 * k + 6]) * inv, __uint_as_float(r[8 * k + 7]) * inv));
          }
        }
      }
    } while (ok && leave(k++));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Gm::TMEM_COLS);
  }
}

// Joins the parts of the blocks that have more than one: out = sum_j w_j O_j / sum_j w_j
// l_j, w_j = 2^(m_j - max m), in ascending j.  A CTA takes 32 rows of a block, a warp D /
// 8 columns of them, a lane a row.
template <int D>
__global__ void __launch_bounds__(256) latent_prefill_merge(const LatentPrefillParams p) {
  using Gm = LatentPrefillGeo<D>;
  constexpr int C = D / 8;  // columns a warp
  const int unit = blockIdx.x / (Gm::BQ / 32), row = (blockIdx.x % (Gm::BQ / 32)) * 32 + (threadIdx.x & 31);
  const int bh = unit / p.nqb, qb = unit - bh * p.nqb, b = bh / p.H, h = bh - b * p.H;
  pdl_wait_primary();
  pdl_launch_dependents();
  int L = p.seq_lens ? load_dependent(p.seq_lens + b) : p.max_len;
  L = L < 0 ? 0 : (L > p.max_len ? p.max_len : L);
  const int q0 = qb * Gm::BQ, nq = min(Gm::BQ, p.q_len - q0);
  const int kv_end = max(0, min(L, L - p.q_len + q0 + nq));
  const int n = prefill_block_parts((kv_end + Gm::BK - 1) / Gm::BK, p.parts);
  if (n <= 1 || row >= nq) return;
  const float kNegInf = -__int_as_float(0x7f800000);
  const size_t slot0 = (size_t)unit * p.parts;
  float M = kNegInf;
  for (int j = 0; j < n; ++j) {
    const float2 ml = __ldcg(p.part_ml + (slot0 + j) * Gm::BQ + row);
    if (ml.y > 0.f || ml.y != ml.y) M = fmaxf(M, ml.x);
  }
  float s[C], den = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) s[c] = 0.f;
  const int c0 = (threadIdx.x >> 5) * C;
  for (int j = 0; j < n; ++j) {
    const float* acc = p.part_acc + ((slot0 + j) * D + c0) * Gm::BQ + row;
    float a[C];
#pragma unroll
    for (int c = 0; c < C; ++c) a[c] = __ldcg(acc + c * Gm::BQ);
    const float2 ml = __ldcg(p.part_ml + (slot0 + j) * Gm::BQ + row);
    const float w = ml.y > 0.f || ml.y != ml.y ? exp2_approx(ml.x - M) : 0.f;
    if (w != 0.f) {
      den += w * ml.y;
#pragma unroll
      for (int c = 0; c < C; ++c) s[c] += w * a[c];
    }
  }
  const float inv = den > 0.f || den != den ? 1.f / den : 0.f;
  uint4* o = reinterpret_cast<uint4*>(p.out + (((size_t)b * p.q_len + q0 + row) * p.H + h) * D + c0);
#pragma unroll
  for (int k = 0; k < C / 8; ++k)
    o[k] = make_uint4(pack_bf16x2(s[8 * k] * inv, s[8 * k + 1] * inv), pack_bf16x2(s[8 * k + 2] * inv, s[8 * k + 3] * inv),
                      pack_bf16x2(s[8 * k + 4] * inv, s[8 * k + 5] * inv),
                      pack_bf16x2(s[8 * k + 6] * inv, s[8 * k + 7] * inv));
}

}  // namespace da
