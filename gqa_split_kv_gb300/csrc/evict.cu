// Entry points of the attention weights and of eviction by them (declared in
// include/decode_attn.h).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/decode_attn.h"
#include "evict_kernel.cuh"
#include "host_util.cuh"
#include "seg_host.cuh"
#include "units.cuh"
#include "weights_kernel.cuh"
#include "weights_tc.cuh"

namespace da {

int take_evict_error_word(unsigned int* flags) { return take_unit_error_word(flags); }

namespace {

// ---------------------------------------------------------------- weights

struct WeightsCall {
  WeightsParams w;
  bool paged, int8;
  int D;
  long long cap;
  void* workspace;
  long long workspace_bytes;
};

constexpr int kWindowRows = 128, kWeightRows = 1024;

struct WeightsShape {
  int rows;                       // of a KV head
  long long slots, score, bytes;  // score: bytes of the scores
};
int weights_shape(int B, int n, int Hq, int Hkv, long long cap, int sms, WeightsShape* s) {
  if (B < 0 || n < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || cap < 0) return DA_ERR_INVALID_ARG;
  const int G = Hq / Hkv;
  if (G > 64 || Hq > 65536 || cap > kMostTokens || product(n, G) > kWeightRows || product(B, Hkv) > 0x3fffffffLL)
    return DA_ERR_UNSUPPORTED;
  s->rows = n * G;
  s->slots = (long long)B * Hkv + 4ll * sms;  // 4 CTAs an SM at most
  const long long tiles = product(B, Hkv, (cap + kTile - 1) / kTile);
  if (tiles > 1LL << 40) return DA_ERR_UNSUPPORTED;
  s->score = s->rows <= 16 ? tiles * score_rows(s->rows) * kTile * 4 : 0;
  s->bytes = s->slots * (s->rows <= 16 ? 16 : kWindowRows) * 8 + s->score;
  return DA_OK;
}

template <int D, bool PAGED, bool INT8, int NT>
int launch_few(WeightsParams w, int sms, cudaStream_t st) {
  using Gm = ScoreGeo<D, INT8, NT>;
  w.s.ctas = Gm::PER_SM * sms;
  w.finish_ctas = 4 * sms;  // few starts; of 16 x <= 8192 tokens: 2 an SM 42.2 us, 3 39.6, 4 38.5, 5 42.0, 8 42.8
  if (int e = allow_smem<weights_score_kernel<D, PAGED, INT8, NT>>(Gm::SMEM)) return e;
  if (int e = launch_dependent(weights_score_kernel<D, PAGED, INT8, NT>, (unsigned)w.s.ctas, Gm::THREADS, Gm::SMEM, st, w))
    return e;
  return launch_dependent(weights_finish_kernel<PAGED>, (unsigned)w.finish_ctas, kFinishThreads, 0, st, w);
}
template <int D, bool PAGED, bool INT8>
int launch_scores(WeightsParams w, int sms, cudaStream_t st) {
  if (w.rows <= 8) return launch_few<D, PAGED, INT8, 1>(w, sms, st);
  if (w.rows <= 16) return launch_few<D, PAGED, INT8, 2>(w, sms, st);
  using Gm = WeightsTcGeo<D>;
  static_assert(Gm::ROWS == kWindowRows, "");
  w.s.ctas = Gm::PER_SM * sms;
  w.timeout_ns = kWaitTimeoutNs;
  if (int e = allow_smem<weights_tc_kernel<D, PAGED, INT8, false>>(Gm::SMEM)) return e;
  if (int e = allow_smem<weights_tc_kernel<D, PAGED, INT8, true>>(Gm::SMEM)) return e;
  const int all = w.rows;
  for (w.row0 = 0; w.row0 < all; w.row0 += kWindowRows) {
    w.rows = all - w.row0 < kWindowRows ? all - w.row0 : kWindowRows;
    if (w.row0 > 0) {  // added to what the windows before have written
      w.prior = w.out;
      w.decay = 1.f;
    }
    if (int e = launch_dependent(weights_tc_kernel<D, PAGED, INT8, false>, (unsigned)w.s.ctas, Gm::THREADS, Gm::SMEM, st, w))
      return e;
    if (int e = launch_dependent(weights_tc_kernel<D, PAGED, INT8, true>, (unsigned)w.s.ctas, Gm::THREADS, Gm::SMEM, st, w))
      return e;
  }
  return DA_OK;
}
template <int D>
int launch_weights(const WeightsCall& c, int sms, cudaStream_t st) {
  return c.paged ? (c.int8 ? launch_scores<D, true, true>(c.w, sms, st) : launch_scores<D, true, false>(c.w, sms, st))
                 : (c.int8 ? launch_scores<D, false, true>(c.w, sms, st) : launch_scores<D, false, false>(c.w, sms, st));
}

int weights_call(WeightsCall& c, float scale, void* stream) {
  WeightsParams& w = c.w;
  SegParams& p = w.s;
  WeightsShape s;
  if (int e = weights_shape(p.B, p.n, p.Hq, p.Hkv, c.cap, 1, &s)) return e;
  if (c.D != 64 && c.D != 128 && c.D != 256) return DA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale) || !std::isfinite(w.decay)) return DA_ERR_INVALID_ARG;
  if (c.paged && (p.page_size <= 0 || p.max_pages < 0 || p.num_pages < 0)) return DA_ERR_INVALID_ARG;
  if (c.paged && p.page_size % 16) return DA_ERR_UNSUPPORTED;
  if (p.B == 0 || c.cap == 0 || (c.paged && p.num_pages == 0)) return DA_OK;
  p.cap = (int)c.cap;
  p.G = p.Hq / p.Hkv;
  if (!p.k || !w.out || (p.n > 0 && !p.q) || !aligned(p.q, 16) || !aligned(p.k, 16) || !aligned(w.k_scale, 4) ||
      !aligned(w.prior, 4) || !aligned(w.out, 4) || !aligned(p.seq_lens, 4) || !aligned(p.page_table, 4) ||
      (c.int8 && !w.k_scale) || (c.paged && (!p.seq_lens || !p.page_table)))
    return DA_ERR_INVALID_ARG;
  const long long cells = product(c.paged ? p.num_pages : p.B, c.paged ? p.page_size : p.ctx, p.Hkv);
  const long long on = product(cells, 4), kn = product(cells, c.D, c.int8 ? 1 : 2), qn = product(p.B, p.n, p.Hq, c.D, 2);
  if (overlap(w.out, on, p.k, kn) || overlap(w.out, on, p.q, qn) || overlap(w.out, on, w.k_scale, on) ||
      (w.prior != w.out && overlap(w.out, on, w.prior, on)))
    return DA_ERR_INVALID_ARG;
  int dev, sms, optin;
  if (current_device(&dev) || device_info(dev, &sms, &optin)) return DA_ERR_CUDA;
  if (int e = weights_shape(p.B, p.n, p.Hq, p.Hkv, c.cap, sms, &s)) return e;
  if (!c.workspace || !aligned(c.workspace, 16) || c.workspace_bytes < s.bytes) return DA_ERR_WORKSPACE;
  for (const void* x : {(const void*)p.k, (const void*)p.q, (const void*)w.out, (const void*)w.prior, (const void*)w.k_scale})
    if (overlap(c.workspace, s.bytes, x, x == p.k ? kn : x == p.q ? qn : on)) return DA_ERR_INVALID_ARG;
  p.rt = 1;
  p.ru = 16;
  w.rows = s.rows;
  p.part_ml = static_cast<float2*>(c.workspace);
  w.scores = reinterpret_cast<float*>(p.part_ml + s.slots * 16);
  p.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return c.D == 64    ? launch_weights<64>(c, sms, st)
         : c.D == 128 ? launch_weights<128>(c, sms, st)
                      : launch_weights<256>(c, sms, st);
}

WeightsCall weights_params(const void* q, const void* k, const float* k_scale, const int* page_table,
                           const int* seq_lens, int batch, int q_len, int num_q_heads, int num_kv_heads, int head_dim,
                           float decay, const float* prior, void* workspace, long long workspace_bytes, float* out) {
  WeightsCall c = {};
  c.w.s.q = static_cast<const __nv_bfloat16*>(q);
  c.w.s.k = static_cast<const __nv_bfloat16*>(k);
  c.w.k_scale = k_scale;
  c.w.s.page_table = page_table;
  c.w.s.seq_lens = seq_lens;
  c.w.s.B = batch;
  c.w.s.n = q_len;
  c.w.s.Hq = num_q_heads;
  c.w.s.Hkv = num_kv_heads;
  c.w.decay = decay;
  c.w.prior = prior;
  c.w.out = out;
  c.D = head_dim;
  c.workspace = workspace;
  c.workspace_bytes = workspace_bytes;
  return c;
}

int weights_contig(WeightsCall c, bool int8, int max_ctx, float scale, void* stream) {
  c.int8 = int8;
  c.w.s.ctx = max_ctx;
  c.cap = max_ctx;
  return weights_call(c, scale, stream);
}
int weights_paged(WeightsCall c, bool int8, int page_size, int max_pages, int num_pages, int max_seq_len, float scale,
                  void* stream) {
  if (max_seq_len < 0) return DA_ERR_INVALID_ARG;
  c.int8 = int8;
  c.paged = true;
  c.w.s.page_size = page_size;
  c.w.s.max_pages = max_pages;
  c.w.s.num_pages = num_pages;
  c.cap = capacity(page_size, max_pages, max_seq_len);
  return weights_call(c, scale, stream);
}

// ---------------------------------------------------------------- eviction

constexpr int kEvictKeys = 48 * 1024;  // 192 KB

int evict_call(EvictParams& p, bool paged, bool int8, int head_dim, long long cap, void* stream) {
  if (p.B < 0 || p.Hkv <= 0 || head_dim <= 0 || cap < 0 || p.keep <= 0 || p.first < 0 || p.recent < 0 ||
      (long long)p.first + p.recent > p.keep)
    return DA_ERR_INVALID_ARG;
  if (paged && (p.slab <= 0 || p.max_pages < 0 || p.num_pages < 0)) return DA_ERR_INVALID_ARG;
  p.row_bytes = head_dim * (int8 ? 1 : 2);
  if (head_dim > 1024 || p.Hkv > 1024 || p.row_bytes % 16 || cap > kMostTokens - 4096 || p.keep > kMostTokens - 4096 ||
      p.out_ctx > kMostTokens ||
      product(p.B, p.Hkv) > 0x7fffffffLL / 1024)
    return DA_ERR_UNSUPPORTED;
  p.in_place = !p.k_out && !p.v_out && !p.ks_out && !p.vs_out && !p.weights_out;
  if (p.B == 0) return DA_OK;
  const bool rows = cap > 0 && (!paged || p.num_pages > 0);
  p.cap = rows ? (int)cap : 0;
  if (!p.kept || !p.new_lens || !aligned(p.kept, 4) || !aligned(p.new_lens, 4) || !aligned(p.seq_lens, 4) ||
      !aligned(p.page_table, 4) || (paged && (!p.seq_lens || (p.max_pages > 0 && !p.page_table))))
    return DA_ERR_INVALID_ARG;
  // (a cache without a token may have no memory: only the outputs have to be whole then)
  if (rows && (!p.k || !p.weights || (int8 && (!p.ks || !p.v != !p.vs)))) return DA_ERR_INVALID_ARG;
  if (!int8 && (p.ks || p.vs || p.ks_out || p.vs_out)) return DA_ERR_INVALID_ARG;
  if (!p.in_place && (!p.k_out || (rows && !p.v != !p.v_out) || p.out_ctx < p.keep ||
                      (int8 && (!p.ks_out || !p.v_out != !p.vs_out))))
    return DA_ERR_INVALID_ARG;
  for (const void* x : {p.k, p.v, p.k_out, p.v_out})
    if (!aligned(x, 16)) return DA_ERR_INVALID_ARG;
  for (const void* x : {p.ks, p.vs, p.weights, p.ks_out, p.vs_out, p.weights_out})
    if (!aligned(x, 4)) return DA_ERR_INVALID_ARG;
  {
    // nothing that is written may be read by the same call otherwise, nor written twice
    const long long cells = product(paged ? p.num_pages : p.B, p.slab, p.Hkv), cn = product(cells, p.row_bytes),
                    sn = product(cells, 4), oc = product(p.B, p.out_ctx, p.Hkv), ocn = product(oc, p.row_bytes),
                    osn = product(oc, 4);
    const void* in[] = {p.k, p.v, p.ks, p.vs, p.weights, p.seq_lens, p.page_table};
    const long long in_bytes[] = {cn, cn, sn, sn, sn, product(p.B, 4), product(p.B, p.max_pages, 4)};
    const void* out[] = {p.kept, p.new_lens, p.k_out, p.v_out, p.ks_out, p.vs_out, p.weights_out};
    const long long out_bytes[] = {product(p.B, p.Hkv, p.keep, 4), product(p.B, 4), ocn, ocn, osn, osn, osn};
    for (int i = 0; i < 7; ++i) {
      for (int j = 0; j < 7; ++j)
        if (overlap(out[i], out_bytes[i], in[j], in_bytes[j])) return DA_ERR_INVALID_ARG;
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out_bytes[i], out[j], out_bytes[j])) return DA_ERR_INVALID_ARG;
    }
    if (p.in_place)
      for (int i = 0; i < 5; ++i)
        for (int j = 0; j < 7; ++j)
          if (i != j && overlap(in[i], in_bytes[i], in[j], in_bytes[j])) return DA_ERR_INVALID_ARG;
  }
  int dev, sms, optin;
  if (current_device(&dev) || device_info(dev, &sms, &optin)) return DA_ERR_CUDA;
  if (p.in_place) {
    p.k_out = p.k;
    p.v_out = p.v;
    p.ks_out = p.ks;
    p.vs_out = p.vs;
    p.weights_out = p.weights;
  }
  const int units = p.B * p.Hkv, tensors = p.v ? 2 : 1, chunks = p.row_bytes / 16;
  p.parts = p.columns = 1;
  if (p.in_place) {
    // only columns of a row may go to different CTAs: 32 bytes at the least
    while (chunks % (2 * p.columns) == 0 && chunks / p.columns >= 4 && (long long)units * tensors * p.columns < 4LL * sms)
      p.columns *= 2;
  } else {
    while (p.parts < 64 && (long long)units * tensors * p.parts < 8LL * sms && (long long)p.keep / (2 * p.parts) * chunks >= kMoveThreads)
      p.parts *= 2;
  }
  const long long grid = (long long)units * (tensors * p.columns * p.parts + 3);
  if (grid > 0x7fffffffLL) return DA_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // a cluster where there are SMs for it and 1024 weights a CTA
  p.cluster = 1;
  while (p.cluster < 8 && (long long)units * p.cluster * 2 <= 4LL * sms && p.cap >= p.cluster * 2 * 1024)
    p.cluster *= 2;
  const int share = p.cap / p.cluster + 1;
  p.keys = share < kEvictKeys ? share : kEvictKeys;
  if (int e = paged ? allow_smem<evict_select_kernel<true>>(kEvictKeys * 4) : allow_smem<evict_select_kernel<false>>(kEvictKeys * 4))
    return e;
  const unsigned ctas = (unsigned)(units * p.cluster);
  if (int e = paged ? launch_clusters(evict_select_kernel<true>, ctas, kEvictThreads, p.keys * 4, p.cluster, st, p)
                    : launch_clusters(evict_select_kernel<false>, ctas, kEvictThreads, p.keys * 4, p.cluster, st, p))
    return e;
  return paged ? launch_dependent(evict_move_kernel<true>, (unsigned)grid, kMoveThreads, 0, st, p)
               : launch_dependent(evict_move_kernel<false>, (unsigned)grid, kMoveThreads, 0, st, p);
}

EvictParams evict_params(void* k, void* v, float* ks, float* vs, float* weights, const int* page_table,
                         const int* seq_lens, int batch, int num_kv_heads, int slab, int max_pages, int num_pages,
                         int keep, int first, int recent, void* k_out, void* v_out, float* ks_out, float* vs_out,
                         float* weights_out, int out_ctx, int* kept, int* new_lens) {
  EvictParams p = {};
  p.k = k;
  p.v = v;
  p.ks = ks;
  p.vs = vs;
  p.weights = weights;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.B = batch;
  p.Hkv = num_kv_heads;
  p.slab = slab;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.keep = keep;
  p.first = first;
  p.recent = recent;
  p.k_out = k_out;
  p.v_out = v_out;
  p.ks_out = ks_out;
  p.vs_out = vs_out;
  p.weights_out = weights_out;
  p.out_ctx = out_ctx;
  p.kept = kept;
  p.new_lens = new_lens;
  return p;
}

}  // namespace
}  // namespace da

using namespace da;

extern "C" long long kv_weights_workspace_bytes(int batch, int q_len, int num_q_heads, int num_kv_heads, int max_len,
                                                int num_sms) {
  int sms = num_sms;
  if (sms <= 0) {
    int dev, optin;
    if (current_device(&dev) || device_info(dev, &sms, &optin)) return -DA_ERR_CUDA;
  }
  WeightsShape s;
  if (int e = weights_shape(batch, q_len, num_q_heads, num_kv_heads, max_len, sms, &s)) return -e;
  return s.bytes;
}

extern "C" int kv_weights_contig(const void* q, const void* k, const int* seq_lens, int batch, int q_len,
                                 int num_q_heads, int num_kv_heads, int head_dim, int max_ctx, float scale, float decay,
                                 const float* prior, void* workspace, long long workspace_bytes, float* out,
                                 void* stream) {
  return weights_contig(weights_params(q, k, nullptr, nullptr, seq_lens, batch, q_len, num_q_heads, num_kv_heads,
                                       head_dim, decay, prior, workspace, workspace_bytes, out),
                        false, max_ctx, scale, stream);
}

extern "C" int kv_weights_paged(const void* q, const void* k_pool, const int* page_table, const int* seq_lens, int batch,
                                int q_len, int num_q_heads, int num_kv_heads, int head_dim, int page_size,
                                int max_pages_per_seq, int num_pages, int max_seq_len, float scale, float decay,
                                const float* prior, void* workspace, long long workspace_bytes, float* out,
                                void* stream) {
  return weights_paged(weights_params(q, k_pool, nullptr, page_table, seq_lens, batch, q_len, num_q_heads, num_kv_heads,
                                      head_dim, decay, prior, workspace, workspace_bytes, out),
                       false, page_size, max_pages_per_seq, num_pages, max_seq_len, scale, stream);
}

extern "C" int kv_weights_int8_contig(const void* q, const void* k_i8, const float* k_scale, const int* seq_lens,
                                      int batch, int q_len, int num_q_heads, int num_kv_heads, int head_dim, int max_ctx,
                                      float scale, float decay, const float* prior, void* workspace,
                                      long long workspace_bytes, float* out, void* stream) {
  return weights_contig(weights_params(q, k_i8, k_scale, nullptr, seq_lens, batch, q_len, num_q_heads, num_kv_heads,
                                       head_dim, decay, prior, workspace, workspace_bytes, out),
                        true, max_ctx, scale, stream);
}

extern "C" int kv_weights_int8_paged(const void* q, const void* k_pool_i8, const float* k_scale_pool,
                                     const int* page_table, const int* seq_lens, int batch, int q_len, int num_q_heads,
                                     int num_kv_heads, int head_dim, int page_size, int max_pages_per_seq, int num_pages,
                                     int max_seq_len, float scale, float decay, const float* prior, void* workspace,
                                     long long workspace_bytes, float* out, void* stream) {
  return weights_paged(weights_params(q, k_pool_i8, k_scale_pool, page_table, seq_lens, batch, q_len, num_q_heads,
                                      num_kv_heads, head_dim, decay, prior, workspace, workspace_bytes, out),
                       true, page_size, max_pages_per_seq, num_pages, max_seq_len, scale, stream);
}

extern "C" int kv_evict_contig(void* k, void* v, float* weights, const int* seq_lens, int batch, int num_kv_heads,
                               int head_dim, int max_ctx, int keep, int first, int recent, void* k_out, void* v_out,
                               float* weights_out, int out_ctx, int* kept, int* new_lens, void* stream) {
  EvictParams p = evict_params(k, v, nullptr, nullptr, weights, nullptr, seq_lens, batch, num_kv_heads, max_ctx, 0, 0,
                               keep, first, recent, k_out, v_out, nullptr, nullptr, weights_out, out_ctx, kept, new_lens);
  return evict_call(p, false, false, head_dim, max_ctx, stream);
}

extern "C" int kv_evict_paged(void* k_pool, void* v_pool, float* weights_pool, const int* page_table,
                              const int* seq_lens, int batch, int num_kv_heads, int head_dim, int page_size,
                              int max_pages_per_seq, int num_pages, int max_seq_len, int keep, int first, int recent,
                              void* k_out, void* v_out, float* weights_out, int out_ctx, int* kept, int* new_lens,
                              void* stream) {
  if (max_seq_len < 0) return DA_ERR_INVALID_ARG;
  EvictParams p = evict_params(k_pool, v_pool, nullptr, nullptr, weights_pool, page_table, seq_lens, batch, num_kv_heads,
                               page_size, max_pages_per_seq, num_pages, keep, first, recent, k_out, v_out, nullptr,
                               nullptr, weights_out, out_ctx, kept, new_lens);
  return evict_call(p, true, false, head_dim, capacity(page_size, max_pages_per_seq, max_seq_len), stream);
}

extern "C" int kv_evict_int8_contig(void* k_i8, void* v_i8, float* k_scale, float* v_scale, float* weights,
                                    const int* seq_lens, int batch, int num_kv_heads, int head_dim, int max_ctx, int keep,
                                    int first, int recent, void* k_out, void* v_out, float* k_scale_out,
                                    float* v_scale_out, float* weights_out, int out_ctx, int* kept, int* new_lens,
                                    void* stream) {
  EvictParams p = evict_params(k_i8, v_i8, k_scale, v_scale, weights, nullptr, seq_lens, batch, num_kv_heads, max_ctx, 0,
                               0, keep, first, recent, k_out, v_out, k_scale_out, v_scale_out, weights_out, out_ctx, kept,
                               new_lens);
  return evict_call(p, false, true, head_dim, max_ctx, stream);
}

extern "C" int kv_evict_int8_paged(void* k_pool_i8, void* v_pool_i8, float* k_scale_pool, float* v_scale_pool,
                                   float* weights_pool, const int* page_table, const int* seq_lens, int batch,
                                   int num_kv_heads, int head_dim, int page_size, int max_pages_per_seq, int num_pages,
                                   int max_seq_len, int keep, int first, int recent, void* k_out, void* v_out,
                                   float* k_scale_out, float* v_scale_out, float* weights_out, int out_ctx, int* kept,
                                   int* new_lens, void* stream) {
  if (max_seq_len < 0) return DA_ERR_INVALID_ARG;
  EvictParams p = evict_params(k_pool_i8, v_pool_i8, k_scale_pool, v_scale_pool, weights_pool, page_table, seq_lens, batch,
                               num_kv_heads, page_size, max_pages_per_seq, num_pages, keep, first, recent, k_out, v_out,
                               k_scale_out, v_scale_out, weights_out, out_ctx, kept, new_lens);
  return evict_call(p, true, true, head_dim, capacity(page_size, max_pages_per_seq, max_seq_len), stream);
}
