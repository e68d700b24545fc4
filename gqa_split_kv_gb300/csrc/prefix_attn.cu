// Entry points of attention behind a shared prefix (declared in include/decode_attn.h).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/decode_attn.h"
#include "host_util.cuh"
#include "prefix_tc.cuh"
#include "seg_host.cuh"
#include "seg_kernel.cuh"
#include "units.cuh"

namespace da {

int take_prefix_error_word(unsigned int* flags) { return take_unit_error_word(flags); }

namespace {

template <int D>
constexpr int tc_rows() { return PrefixTcGeo<D>::ROWS; }
int tc_rows(int D) { return D == 64 ? tc_rows<64>() : D == 128 ? tc_rows<128>() : tc_rows<256>(); }

constexpr int kFewRows = 64;  // of a KV head: those that may read the prefix in seg_kernel

// What a call of these sizes launches.
struct PrefixShape {
  int ru, rt, rt_prefix, ctas;  // seg_kernel's
  int splits, row_blocks;      // prefix_tc_kernel's: the most parts that a prefix's keys may have
  long long slots, rows, tc_ml, bytes;  // tc_ml: bytes of the parts' (m, l)
};

int prefix_shape(int B, int n, int Hq, int Hkv, int D, int sms, PrefixShape* s) {
  if (B < 0 || n < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv) return DA_ERR_INVALID_ARG;
  if (D != 64 && D != 128 && D != 256) return DA_ERR_UNSUPPORTED;
  const int G = Hq / Hkv;
  if (G > 64 || Hq > 65536 || product(B, n, Hq) > 0x7fffffffLL / 16) return DA_ERR_UNSUPPORTED;
  s->rows = (long long)B * n * G;
  s->ru = seg_unit_rows((long long)n * G, D);
  s->rt = (int)(((long long)n * G + s->ru - 1) / s->ru);
  s->ctas = seg_ctas(s->ru, D, sms);
  // few rows: the prefix may go through seg_kernel, as more units of a head
  s->rt_prefix = s->rows <= kFewRows ? (int)((s->rows + s->ru - 1) / s->ru) : 0;
  s->row_blocks = (int)((s->rows + tc_rows(D) - 1) / tc_rows(D));
  const long long units = product(Hkv, s->row_blocks);
  s->splits = s->rows <= 16 || units == 0 ? 0 : units >= sms ? 1 : (int)(sms / units);
  s->slots = (long long)Hkv * s->rt_prefix + (long long)B * Hkv * s->rt + s->ctas;
  s->tc_ml = (s->splits * product(Hkv, s->rows, 8) + 15) / 16 * 16;
  s->bytes = seg_partial_bytes(s->slots, s->ru, D) + s->tc_ml + s->splits * product(Hkv, s->rows, D * 4);
  return DA_OK;
}

struct PrefixCall {
  SegParams p;
  bool paged;
  int D;
  void* workspace;
  long long workspace_bytes;
  long long cap;
};

// The prefix's part on the tensor cores.
template <int D>
int launch_tc(const PrefixCall& c, const PrefixTcParams& base, cudaStream_t st) {
  using Gm = PrefixTcGeo<D>;
  if (int e = allow_smem<prefix_tc_kernel<D>>(Gm::SMEM)) return e;
  if (Gm::NQT == 2) {
    // the softmax warpgroups raise their registers out of what the launch gave the CTA; a build
    // whose per-thread count is below the split would wait for ever, so it is refused
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_relaxed) == 0) {
      cudaFuncAttributes fa;
      if (cudaFuncGetAttributes(&fa, prefix_tc_kernel<D>) != cudaSuccess) {
        cudaGetLastError();
        return DA_ERR_CUDA;
      }
      regs.store(fa.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) * Gm::NTHREADS < Gm::REG_POOL_NEEDED) return DA_ERR_UNSUPPORTED;
  }
  PrefixTcParams t = base;
  const cuuint64_t row = (cuuint64_t)t.Hkv * D * 2;
  const cuuint64_t rows = c.paged ? t.page_size : t.P, pages = c.paged ? t.num_pages : 1;
  int rk = Gm::BK;
  if (c.paged)
    while (t.page_size % rk) rk /= 2;
  const int rv = rk < Gm::VKEYS ? rk : Gm::VKEYS;
  for (t.rk_log2 = 0; 1 << t.rk_log2 < rk;) ++t.rk_log2;
  for (t.rv_log2 = 0; 1 << t.rv_log2 < rv;) ++t.rv_log2;
  const cuuint64_t dims[5] = {64, rows, D / 64, (cuuint64_t)t.Hkv, pages}, strides[4] = {row, 128, D * 2, row * rows};
  const cuuint32_t box_k[5] = {64, (cuuint32_t)rk, 1, 1, 1}, box_v[5] = {64, (cuuint32_t)rv, 1, 1, 1};
  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  if (int e = encode_map_t(&t.tm_k, bf16, sw, c.paged ? c.p.k : c.p.kp, 5, dims, strides, box_k)) return e;
  if (int e = encode_map_t(&t.tm_v, bf16, sw, c.paged ? c.p.v : c.p.vp, 5, dims, strides, box_v)) return e;
  const long long grid = product(t.row_blocks, t.splits, t.Hkv);
  if (grid > 0x7fffffffLL) return DA_ERR_UNSUPPORTED;
  return launch_dependent(prefix_tc_kernel<D>, (unsigned)grid, Gm::NTHREADS, Gm::SMEM, st, t);
}

// Whether the prefix goes through seg_kernel: up to 16 rows, and up to 64 where its tiles of 64 tokens and 8 or 16 rows
// are at most half as many as the CTAs, so that the call takes one kernel less: 32 rows of 8 heads of 128 after 200 tokens
// 10.7 -> 9.5 us, after 512 (256 tiles of 608 CTAs) 11.0 -> 10.4; after 1024 (512) it would be 11.7 -> 12.1.
bool prefix_through_seg(const PrefixShape& s, int Hkv, int P) {
  return s.rows <= 16 || (s.rt_prefix && product(Hkv, s.rt_prefix, (P + kTile - 1) / kTile) * 2 <= s.ctas);
}

template <int D>
int launch_prefix(PrefixCall& c, const PrefixShape& s, int sms, cudaStream_t st) {
  SegParams& p = c.p;
  if (!prefix_through_seg(s, p.Hkv, p.base)) p.rt_prefix = 0;
  if (!p.rt_prefix && p.base > 0) {
    PrefixTcParams t = {};
    t.q = p.q;
    t.seq_lens = p.seq_lens;
    t.prefix_table = c.paged ? p.prefix_table : nullptr;
    t.o = const_cast<float*>(p.tc_o);
    t.ml = const_cast<float2*>(p.tc_ml);
    t.B = p.B;
    t.n = p.n;
    t.Hq = p.Hq;
    t.Hkv = p.Hkv;
    t.G = p.G;
    t.P = p.base;
    t.cap = p.cap;
    t.page_size = p.page_size;
    t.num_pages = p.num_pages;
    t.row_blocks = s.row_blocks;
    // As many parts as there is room for, of whole tiles and alike.  A CTA of the prefix's takes an SM for itself: where the
    // rests can be no more than fill half of the SMs, those stay free for them, if that makes the parts no more than 3
    // times 128 keys longer (a second turn of starts costs as much).  8 x (P + <= 256) tokens, 64/8 heads of 128: P = 2048
    // 18.6 -> 13.3 us, 8192 23.3 -> 19.8, while 32768 would be 38.4 -> 44.3; 24/4 heads of 256, 2048: 22.8 -> 14.1.
    const int tiles = (p.base + PrefixTcGeo<D>::BK - 1) / PrefixTcGeo<D>::BK;
    const long long rests = product(p.B, p.Hkv, p.rt, seg_tiles(p.cap, p.cap, p.base & ~15));
    const long long beside = ((rests < s.ctas ? rests : s.ctas) + s.ctas / sms - 1) / (s.ctas / sms);
    const long long room = (sms - beside) / product(s.row_blocks, p.Hkv);  // parts next to the rests
    int each = (tiles + s.splits - 1) / s.splits;
    if (beside <= sms / 2 && room >= 1 && room < s.splits) {
      const int longer = (int)((tiles + room - 1) / room);
      if ((longer - each) * PrefixTcGeo<D>::BK <= 3 * 128) each = longer;
    }
    t.splits = (tiles + each - 1) / each;
    t.scale_log2 = p.scale_log2;
    t.timeout_ns = kWaitTimeoutNs;
    p.slabs = t.splits;
    p.beside = 1;
    if (int e = launch_tc<D>(c, t, st)) return e;
  }
  const bool edges = p.n > 1 || p.rt_prefix > 0;
  if (int e = c.paged ? (edges ? launch_seg<D, true, kSegEdges>(p, st) : launch_seg<D, true, kSegRange>(p, st))
                      : (edges ? launch_seg<D, false, kSegEdges>(p, st) : launch_seg<D, false, kSegRange>(p, st)))
    return e;
  return launch_dependent(seg_merge_prefix_kernel<D>,
                          (unsigned)(((long long)p.B * p.n * p.Hq + kMergeThreads / 32 - 1) / (kMergeThreads / 32)),
                          kMergeThreads, 0, st, p);
}

int prefix_call(PrefixCall& c, float scale, void* stream) {
  SegParams& p = c.p;
  PrefixShape s;
  int dev, sms, optin;
  if (int e = prefix_shape(p.B, p.n, p.Hq, p.Hkv, c.D, 1, &s)) return e;
  if (p.base < 0 || c.cap < 0 || !std::isfinite(scale)) return DA_ERR_INVALID_ARG;
  if (c.cap > kMostTokens) return DA_ERR_UNSUPPORTED;
  if (c.paged && (p.page_size <= 0 || p.max_pages < 0 || p.num_pages < 0)) return DA_ERR_INVALID_ARG;
  if (c.paged && p.page_size % 16) return DA_ERR_UNSUPPORTED;
  if (p.B == 0 || p.n == 0) return DA_OK;
  p.cap = (int)c.cap;
  if (p.base > p.cap) p.base = p.cap;
  p.G = p.Hq / p.Hkv;
  if (!p.q || !p.out || !aligned(p.q, 16) || !aligned(p.out, 16) || !aligned(p.seq_lens, 4) || !aligned(p.k, 16) ||
      !aligned(p.v, 16) || !aligned(p.kp, 16) || !aligned(p.vp, 16) || !aligned(p.page_table, 4) ||
      !aligned(p.prefix_table, 4))
    return DA_ERR_INVALID_ARG;
  const long long on = product(p.B, p.n, p.Hq, c.D, 2), row = product(p.Hkv, c.D, 2);
  const long long cn = c.paged ? product(p.num_pages, p.page_size, row) : product(p.B, p.ctx, row);
  if (c.paged) {
    if (!p.seq_lens || (p.max_pages > 0 && !p.page_table) || (p.base > 0 && !p.prefix_table) || (cn > 0 && (!p.k || !p.v)))
      return DA_ERR_INVALID_ARG;
    if (p.num_pages == 0) p.base = p.cap = 0;  // no token: zeros
  } else if ((cn > 0 && (!p.k || !p.v)) || (p.base > 0 && (!p.kp || !p.vp))) {
    return DA_ERR_INVALID_ARG;
  }
  const long long pn = c.paged ? 0 : product(p.base, row);
  for (const void* src : {(const void*)p.k, (const void*)p.v})
    if (overlap(p.out, on, src, cn)) return DA_ERR_INVALID_ARG;
  if (overlap(p.out, on, p.q, on) || overlap(p.out, on, p.kp, pn) || overlap(p.out, on, p.vp, pn))
    return DA_ERR_INVALID_ARG;
  if (current_device(&dev) || device_info(dev, &sms, &optin)) return DA_ERR_CUDA;
  if (int e = prefix_shape(p.B, p.n, p.Hq, p.Hkv, c.D, sms, &s)) return e;
  if (!c.workspace || !aligned(c.workspace, 16) || c.workspace_bytes < s.bytes) return DA_ERR_WORKSPACE;
  if (overlap(c.workspace, s.bytes, p.out, on)) return DA_ERR_INVALID_ARG;
  p.rt = s.rt;
  p.rt_prefix = s.rt_prefix;
  p.ctas = s.ctas;
  p.ru = s.ru;
  seg_partials(p, c.workspace, s.slots, c.D);
  p.tc_ml = p.part_ml + s.slots * s.ru;
  p.tc_o = reinterpret_cast<const float*>(reinterpret_cast<const char*>(p.tc_ml) + s.tc_ml);
  p.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return c.D == 64    ? launch_prefix<64>(c, s, sms, st)
         : c.D == 128 ? launch_prefix<128>(c, s, sms, st)
                      : launch_prefix<256>(c, s, sms, st);
}

PrefixCall prefix_params(const void* q, const void* k, const void* v, const int* seq_lens, int batch, int q_len,
                         int num_q_heads, int num_kv_heads, int head_dim, int prefix_len, void* workspace,
                         long long workspace_bytes, void* out) {
  PrefixCall c = {};
  c.p.q = static_cast<const __nv_bfloat16*>(q);
  c.p.k = static_cast<const __nv_bfloat16*>(k);
  c.p.v = static_cast<const __nv_bfloat16*>(v);
  c.p.seq_lens = seq_lens;
  c.p.out = static_cast<__nv_bfloat16*>(out);
  c.p.B = batch;
  c.p.n = q_len;
  c.p.Hq = num_q_heads;
  c.p.Hkv = num_kv_heads;
  c.p.base = prefix_len;
  c.D = head_dim;
  c.workspace = workspace;
  c.workspace_bytes = workspace_bytes;
  return c;
}

}  // namespace
}  // namespace da

using namespace da;

extern "C" long long prefix_attn_workspace_bytes(int batch, int q_len, int num_q_heads, int num_kv_heads, int head_dim,
                                                 int num_sms) {
  int sms = num_sms;
  if (sms <= 0) {
    int dev, optin;
    if (current_device(&dev) || device_info(dev, &sms, &optin)) return -DA_ERR_CUDA;
  }
  PrefixShape s;
  if (int e = prefix_shape(batch, q_len, num_q_heads, num_kv_heads, head_dim, sms, &s)) return -e;
  return s.bytes;
}

extern "C" int prefix_attn_contig(const void* q, const void* k_prefix, const void* v_prefix, const void* k, const void* v,
                                  const int* seq_lens, int batch, int q_len, int num_q_heads, int num_kv_heads,
                                  int head_dim, int prefix_len, int max_ctx, float scale, void* workspace,
                                  long long workspace_bytes, void* out, void* stream) {
  if (max_ctx < 0 || prefix_len < 0) return DA_ERR_INVALID_ARG;
  PrefixCall c = prefix_params(q, k, v, seq_lens, batch, q_len, num_q_heads, num_kv_heads, head_dim, prefix_len,
                               workspace, workspace_bytes, out);
  c.p.kp = static_cast<const __nv_bfloat16*>(k_prefix);
  c.p.vp = static_cast<const __nv_bfloat16*>(v_prefix);
  c.p.ctx = max_ctx;
  c.cap = (long long)prefix_len + max_ctx;
  return prefix_call(c, scale, stream);
}

extern "C" int prefix_attn_paged(const void* q, const void* k_pool, const void* v_pool, const int* prefix_table,
                                 int prefix_len, const int* page_table, const int* seq_lens, int batch, int q_len,
                                 int num_q_heads, int num_kv_heads, int head_dim, int page_size, int max_pages_per_seq,
                                 int num_pages, int max_seq_len, float scale, void* workspace,
                                 long long workspace_bytes, void* out, void* stream) {
  if (max_seq_len < 0) return DA_ERR_INVALID_ARG;
  PrefixCall c = prefix_params(q, k_pool, v_pool, seq_lens, batch, q_len, num_q_heads, num_kv_heads, head_dim,
                               prefix_len, workspace, workspace_bytes, out);
  c.paged = true;
  c.p.prefix_table = prefix_table;
  c.p.page_table = page_table;
  c.p.page_size = page_size;
  c.p.max_pages = max_pages_per_seq;
  c.p.num_pages = num_pages;
  c.cap = capacity(page_size, max_pages_per_seq, max_seq_len);
  return prefix_call(c, scale, stream);
}
