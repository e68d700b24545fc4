// Entry points of attention over selected blocks of a cache (declared in include/decode_attn.h).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/decode_attn.h"
#include "block_select.cuh"
#include "host_util.cuh"
#include "seg_host.cuh"
#include "units.cuh"

namespace da {

int take_sparse_error_word(unsigned int* flags) { return take_unit_error_word(flags); }

namespace {

// ---------------------------------------------------------------- mean keys

int means_call(MeansParams& p, bool paged, long long cap, cudaStream_t st) {
  if (p.B < 0 || p.n < 0 || p.Hkv <= 0 || p.D <= 0 || cap < 0 || p.block <= 0 || p.max_blocks < 0)
    return DA_ERR_INVALID_ARG;
  if (p.D % 8 || p.D > 1024 || p.Hkv > 1024 || cap > kMostTokens - p.block) return DA_ERR_UNSUPPORTED;
  if (paged && (p.page_size <= 0 || p.max_pages < 0 || p.num_pages < 0)) return DA_ERR_INVALID_ARG;
  if (p.block > 65536 || (paged && product(p.num_pages, p.page_size) > 0xffffffffLL)) return DA_ERR_UNSUPPORTED;
  // tokens past the last block have no mean
  if (cap > (long long)p.max_blocks * p.block) return DA_ERR_INVALID_ARG;
  if (p.B == 0 || p.n == 0 || cap == 0 || (paged && p.num_pages == 0)) return DA_OK;
  p.cap = (int)cap;
  if (!p.k || !p.means || !aligned(p.k, 16) || !aligned(p.means, 16) || !aligned(p.seq_lens, 4) ||
      !aligned(p.page_table, 4) || (paged && (!p.seq_lens || !p.page_table)))
    return DA_ERR_INVALID_ARG;
  const long long kn = product(paged ? p.num_pages : p.B, paged ? p.page_size : p.ctx, p.Hkv, p.D, 2);
  if (overlap(p.means, product(p.B, p.Hkv, p.max_blocks, p.D, 2), p.k, kn)) return DA_ERR_INVALID_ARG;
  int dev, sms, optin;
  if (current_device(&dev) || device_info(dev, &sms, &optin)) return DA_ERR_CUDA;
  const long long touched = (p.n - 1ll) / p.block + 2, total = (cap + p.block - 1) / p.block;
  p.touched = (int)(touched < total ? touched : total);
  // few blocks: shares of 128 bytes of their rows at the least, until there are 4 CTAs an SM
  const int chunks = p.Hkv * p.D / 8;
  p.shares = (chunks + kMeansThreads - 1) / kMeansThreads;
  while (chunks / (2 * p.shares) >= 8 && (long long)p.B * p.touched * p.shares < 4LL * sms) p.shares *= 2;
  const long long grid = product(p.B, p.touched, p.shares);
  if (grid > 0x7fffffffLL) return DA_ERR_UNSUPPORTED;
  return paged ? launch_dependent(block_means_kernel<true>, (unsigned)grid, kMeansThreads, 0, st, p)
               : launch_dependent(block_means_kernel<false>, (unsigned)grid, kMeansThreads, 0, st, p);
}

MeansParams means_params(const void* k, const int* seq_lens, int batch, int q_len, int num_kv_heads, int head_dim,
                         int block_size, int max_blocks, void* means) {
  MeansParams p = {};
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.seq_lens = seq_lens;
  p.means = static_cast<__nv_bfloat16*>(means);
  p.B = batch;
  p.n = q_len;
  p.Hkv = num_kv_heads;
  p.D = head_dim;
  p.block = block_size;
  p.max_blocks = max_blocks;
  return p;
}

// ---------------------------------------------------------------- selection

template <int D, int THREADS>
int launch_select_by(const SelectParams& p, long long units, cudaStream_t st) {
  if (int e = allow_smem<block_select_kernel<D, THREADS>>(200 * 1024)) return e;
  return launch_clusters(block_select_kernel<D, THREADS>, (unsigned)(units * p.cluster), THREADS,
                         select_smem(p.qt, p.max_blocks), p.cluster, st, p);
}
template <int D>
int launch_select(const SelectParams& p, long long units, int sms, cudaStream_t st) {
  // a CTA's time is its chain of steps; with several rounds of CTAs and no more than 4 steps of 8 blocks a warp,
  // twice as many small ones run at once
  if (units > 2LL * sms && p.max_blocks <= 4 * 8 * 4) return launch_select_by<D, kSelectThreads / 2>(p, units, st);
  return launch_select_by<D, kSelectThreads>(p, units, st);
}

// Heads that a call of this family takes.
int check_heads(int B, int n, int Hq, int Hkv, int D) {
  if (B < 0 || n < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv) return DA_ERR_INVALID_ARG;
  if ((D != 64 && D != 128 && D != 256) || Hq / Hkv > 64 || Hq > 65536 || product(B, n, Hq) > 0x7fffffffLL / 16)
    return DA_ERR_UNSUPPORTED;
  return DA_OK;
}

// ---------------------------------------------------------------- attention

struct SparseCall {
  SegParams p;
  bool paged;
  int D;
  long long cap;
};

template <int D>
int launch_sparse(const SparseCall& c, cudaStream_t st) {
  return c.paged ? launch_seg<D, true, kSegBlocks>(c.p, st) : launch_seg<D, false, kSegBlocks>(c.p, st);
}

int sparse_call(SparseCall& c, float scale, cudaStream_t st) {
  SegParams& p = c.p;
  if (int e = check_heads(p.B, p.n, p.Hq, p.Hkv, c.D)) return e;
  if (c.cap < 0 || p.pick <= 0 || p.block <= 0 || !std::isfinite(scale)) return DA_ERR_INVALID_ARG;
  if (c.paged && (p.page_size <= 0 || p.max_pages < 0 || p.num_pages < 0)) return DA_ERR_INVALID_ARG;
  if (p.block % 16 || p.block > 65536 || (long long)p.pick * p.block > kMostTokens ||
      c.cap > kMostTokens - p.block || (c.paged && p.page_size % 16))
    return DA_ERR_UNSUPPORTED;
  if (p.B == 0 || p.n == 0) return DA_OK;
  p.cap = c.paged && p.num_pages == 0 ? 0 : (int)c.cap;
  p.G = p.Hq / p.Hkv;
  const long long on = product(p.B, p.n, p.Hq, c.D, 2), bn = product(p.B, p.n, p.Hkv, p.pick, 4);
  const long long cn = product(c.paged ? p.num_pages : p.B, c.paged ? p.page_size : p.ctx, p.Hkv, c.D, 2);
  if (!p.q || !p.out || !p.blocks || !aligned(p.q, 16) || !aligned(p.out, 16) || !aligned(p.blocks, 4) ||
      !aligned(p.k, 16) || !aligned(p.v, 16) || !aligned(p.seq_lens, 4) || !aligned(p.page_table, 4) ||
      (cn > 0 && (!p.k || !p.v)) || (c.paged && (!p.seq_lens || (p.max_pages > 0 && !p.page_table))))
    return DA_ERR_INVALID_ARG;
  if (overlap(p.out, on, p.q, on) || overlap(p.out, on, p.k, cn) || overlap(p.out, on, p.v, cn) ||
      overlap(p.out, on, p.blocks, bn))
    return DA_ERR_INVALID_ARG;
  int dev, sms, optin;
  if (current_device(&dev) || device_info(dev, &sms, &optin)) return DA_ERR_CUDA;
  p.ru = seg_unit_rows(p.G, c.D);
  p.rt = (p.G + p.ru - 1) / p.ru;
  const long long units = product(p.B, p.n, p.Hkv, p.rt), room = seg_ctas(p.ru, c.D, sms);
  if (units > 0x7fffffffLL) return DA_ERR_UNSUPPORTED;
  // CTAs a unit: as many as make the rounds over the card shortest, a unit's fixed work counting as 2 tiles
  const long long tiles = (p.pick * p.block + kTile - 1) / kTile;
  long long best = 0;
  for (int k = 1; k <= kSegCluster && k <= tiles; k *= 2) {
    const long long at_once = room / k, cost = (units + at_once - 1) / at_once * ((tiles + k - 1) / k + 2);
    if (k > 1 && cost >= best) continue;
    best = cost;
    p.cluster = k;
    p.ctas = (int)((units < at_once ? units : at_once) * k);
  }
  p.scale_log2 = scale * 1.4426950408889634f;
  return c.D == 64 ? launch_sparse<64>(c, st) : c.D == 128 ? launch_sparse<128>(c, st) : launch_sparse<256>(c, st);
}

SparseCall sparse_params(const void* q, const void* k, const void* v, const int* blocks, const int* seq_lens, int batch,
                         int q_len, int num_q_heads, int num_kv_heads, int head_dim, int block_size, int n_select,
                         void* out) {
  SparseCall c = {};
  c.p.q = static_cast<const __nv_bfloat16*>(q);
  c.p.k = static_cast<const __nv_bfloat16*>(k);
  c.p.v = static_cast<const __nv_bfloat16*>(v);
  c.p.blocks = blocks;
  c.p.seq_lens = seq_lens;
  c.p.out = static_cast<__nv_bfloat16*>(out);
  c.p.B = batch;
  c.p.n = q_len;
  c.p.Hq = num_q_heads;
  c.p.Hkv = num_kv_heads;
  c.p.block = block_size;
  c.p.pick = n_select;
  c.D = head_dim;
  return c;
}

}  // namespace
}  // namespace da

using namespace da;

extern "C" int block_means_contig(const void* k, const int* seq_lens, int batch, int q_len, int num_kv_heads,
                                  int head_dim, int max_ctx, int block_size, int max_blocks, void* means, void* stream) {
  MeansParams p = means_params(k, seq_lens, batch, q_len, num_kv_heads, head_dim, block_size, max_blocks, means);
  p.ctx = max_ctx;
  return means_call(p, false, max_ctx, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int block_means_paged(const void* k_pool, const int* page_table, const int* seq_lens, int batch, int q_len,
                                 int num_kv_heads, int head_dim, int page_size, int max_pages_per_seq, int num_pages,
                                 int max_seq_len, int block_size, int max_blocks, void* means, void* stream) {
  if (max_seq_len < 0) return DA_ERR_INVALID_ARG;
  MeansParams p = means_params(k_pool, seq_lens, batch, q_len, num_kv_heads, head_dim, block_size, max_blocks, means);
  p.page_table = page_table;
  p.page_size = page_size;
  p.max_pages = max_pages_per_seq;
  p.num_pages = num_pages;
  return means_call(p, true, capacity(page_size, max_pages_per_seq, max_seq_len), reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int block_select(const void* q, const void* means, const int* seq_lens, int batch, int q_len, int num_q_heads,
                            int num_kv_heads, int head_dim, int block_size, int max_blocks, int n_select, int first,
                            int recent, int* out, void* stream) {
  if (int e = check_heads(batch, q_len, num_q_heads, num_kv_heads, head_dim)) return e;
  if (block_size <= 0 || max_blocks < 0 || n_select <= 0 || first < 0 || recent < 1 || (long long)first + recent > n_select)
    return DA_ERR_INVALID_ARG;
  if (block_size > 65536 || max_blocks > kSelectBlocks || n_select > kMostTokens) return DA_ERR_UNSUPPORTED;
  if (batch == 0 || q_len == 0) return DA_OK;
  const long long qn = product(batch, q_len, num_q_heads, head_dim, 2), mn = product(batch, num_kv_heads, max_blocks, head_dim, 2),
                  on = product(batch, q_len, num_kv_heads, n_select, 4);
  if (!q || !out || (mn > 0 && !means) || !aligned(q, 16) || !aligned(means, 16) || !aligned(out, 4) || !aligned(seq_lens, 4))
    return DA_ERR_INVALID_ARG;
  if (overlap(out, on, q, qn) || overlap(out, on, means, mn)) return DA_ERR_INVALID_ARG;
  int dev, sms, optin;
  if (current_device(&dev) || device_info(dev, &sms, &optin)) return DA_ERR_CUDA;
  SelectParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.means = static_cast<const __nv_bfloat16*>(means);
  p.seq_lens = seq_lens;
  p.out = out;
  p.B = batch;
  p.n = q_len;
  p.Hq = num_q_heads;
  p.Hkv = num_kv_heads;
  p.G = num_q_heads / num_kv_heads;
  p.cap = (int)((long long)max_blocks * block_size);
  p.block = block_size;
  p.max_blocks = max_blocks;
  p.pick = n_select;
  p.first = first;
  p.recent = recent;
  // as many tokens as fill the MMA's 16 rows, while their scores leave room for several CTAs an SM
  p.qt = p.G >= 16 ? 1 : 16 / p.G;
  p.qt = p.qt < q_len ? p.qt : q_len;
  while (p.qt > 1 && select_smem(p.qt, max_blocks) > 96 * 1024) p.qt /= 2;
  const long long units = product(batch, num_kv_heads, (q_len + p.qt - 1) / p.qt);
  // few queries over many blocks: the CTAs of a cluster share the scores, down to two steps a warp
  p.cluster = 1;
  while (p.cluster < 8 && units * p.cluster * 2 <= 4LL * sms && max_blocks >= 2 * p.cluster * 2 * kSelectThreads / 32 * 8)
    p.cluster *= 2;
  if (units * p.cluster > 0x7fffffffLL) return DA_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return head_dim == 64    ? launch_select<64>(p, units, sms, st)
         : head_dim == 128 ? launch_select<128>(p, units, sms, st)
                           : launch_select<256>(p, units, sms, st);
}

extern "C" int sparse_attn_contig(const void* q, const void* k, const void* v, const int* blocks, const int* seq_lens,
                                  int batch, int q_len, int num_q_heads, int num_kv_heads, int head_dim, int max_ctx,
                                  int block_size, int n_select, float scale, void* out, void* stream) {
  SparseCall c = sparse_params(q, k, v, blocks, seq_lens, batch, q_len, num_q_heads, num_kv_heads, head_dim, block_size,
                               n_select, out);
  c.p.ctx = max_ctx;
  c.cap = max_ctx;
  return sparse_call(c, scale, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int sparse_attn_paged(const void* q, const void* k_pool, const void* v_pool, const int* blocks,
                                 const int* page_table, const int* seq_lens, int batch, int q_len, int num_q_heads,
                                 int num_kv_heads, int head_dim, int page_size, int max_pages_per_seq, int num_pages,
                                 int max_seq_len, int block_size, int n_select, float scale, void* out,
                                 void* stream) {
  if (max_seq_len < 0) return DA_ERR_INVALID_ARG;
  SparseCall c = sparse_params(q, k_pool, v_pool, blocks, seq_lens, batch, q_len, num_q_heads, num_kv_heads, head_dim,
                               block_size, n_select, out);
  c.paged = true;
  c.p.page_table = page_table;
  c.p.page_size = page_size;
  c.p.max_pages = max_pages_per_seq;
  c.p.num_pages = num_pages;
  c.cap = capacity(page_size, max_pages_per_seq, max_seq_len);
  return sparse_call(c, scale, reinterpret_cast<cudaStream_t>(stream));
}
