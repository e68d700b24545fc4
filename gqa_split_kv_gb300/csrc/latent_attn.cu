// Entry points of latent attention (declared in include/decode_attn.h): the absorbed
// form over a contiguous or paged latent cache, and the prefill over expanded keys and
// values.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/decode_attn.h"
#include "device_error.cuh"
#include "host_util.cuh"
#include "latent_kernel.cuh"
#include "latent_prefill.cuh"

namespace da {

int take_latent_error_word(unsigned int* flags) { return take_unit_error_word(flags); }

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Rows of a tile: the smallest built size that holds them all, else tiles of 64.
int latent_tile_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

template <typename K>
int allow_smem(K kern, int bytes, bool (&done)[kMaxDevices], int dev) {
  std::lock_guard<std::mutex> lk(g_mu);
  if (done[dev]) return DA_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
      cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
          cudaSuccess) {
    cudaGetLastError();
    return DA_ERR_UNSUPPORTED;
  }
  done[dev] = true;
  return DA_OK;
}

template <int R, int N, bool PAGED>
int launch_latent(const LatentParams& prm, int sms, int dev, cudaStream_t st) {
  using Gm = LatentGeo<R, N>;
  static bool split_done[kMaxDevices] = {false}, combine_done[kMaxDevices] = {false};
  const long long items = (long long)prm.B * prm.rows * (R / 128);  // of the combine kernel
  if (prm.B > Gm::MAX_BATCH || items > 0x7fffffffLL) return DA_ERR_UNSUPPORTED;
  if (int e = allow_smem(latent_kernel<R, N, PAGED>, 227 * 1024, split_done, dev)) return e;
  if (int e = allow_smem(latent_combine_kernel<R>, 227 * 1024, combine_done, dev)) return e;
  // one CTA a range, and no more ranges than the line has units
  const long long units =
      ((long long)prm.B * prm.U * ((prm.max_len + kBlockTokens - 1) / kBlockTokens + 3 + kLatentGap)) / kRangeQuantum + 1;
  if (int e = launch_dependent(latent_kernel<R, N, PAGED>, (unsigned)(prm.ranges < units ? prm.ranges : units),
                               Gm::NTHREADS, (size_t)Gm::SMEM, st, prm))
    return e;
  const LatentCombineParams c = {prm.part_acc, prm.part_ml, prm.out, prm.seq_lens, prm.B,
                                 prm.rows,     prm.U,       N,       prm.ranges,   prm.max_len};
  // items go a warp at a time, those of long runs a CTA at a time
  return launch_dependent(latent_combine_kernel<R>, (unsigned)(items < sms ? items : sms), LatentCombineGeo::NTHREADS,
                          (size_t)LatentCombineGeo::smem_bytes(prm.ranges, prm.B), st, c);
}

template <int R>
int launch_latent_rows(const LatentParams& prm, int N, bool paged, int sms, int dev, cudaStream_t st) {
  if (N == 16)
    return paged ? launch_latent<R, 16, true>(prm, sms, dev, st) : launch_latent<R, 16, false>(prm, sms, dev, st);
  if (N == 32)
    return paged ? launch_latent<R, 32, true>(prm, sms, dev, st) : launch_latent<R, 32, false>(prm, sms, dev, st);
  return paged ? launch_latent<R, 64, true>(prm, sms, dev, st) : launch_latent<R, 64, false>(prm, sms, dev, st);
}

template <int R>
int latent_batch_limit(int N) {
  return N == 16 ? LatentGeo<R, 16>::MAX_BATCH : N == 32 ? LatentGeo<R, 32>::MAX_BATCH : LatentGeo<R, 64>::MAX_BATCH;
}

int latent_shape(int batch, int q_len, int num_heads, int latent_dim) {
  if (batch < 0 || q_len < 1 || q_len > DA_MAX_QLEN || num_heads < 1) return DA_ERR_INVALID_ARG;
  if (latent_dim != 128 && latent_dim != 256 && latent_dim != 512) return DA_ERR_UNSUPPORTED;
  if (num_heads > DA_MAX_LATENT_HEADS) return DA_ERR_UNSUPPORTED;
  return DA_OK;
}

long long latent_part_rows(int rows, int sms) { return 2LL * sms * latent_tile_rows(rows); }

// partials, their (m, l), and the list of pieces
long long latent_workspace(int B, int rows, int R, int sms) {
  const int N = latent_tile_rows(rows);
  return latent_part_rows(rows, sms) * (R * 4 + 8) + (sms + (long long)B * ((rows + N - 1) / N)) * 16;
}

int latent_call(bool paged, const void* q, const void* cache, const int* page_table, const int* seq_lens, int B,
                int q_len, int H, int R, long long max_len, int page_size, int max_pages, int num_pages, float scale,
                void* workspace, long long workspace_bytes, void* out, cudaStream_t st) {
  if (int e = latent_shape(B, q_len, H, R)) return e;
  if (!std::isfinite(scale)) return DA_ERR_INVALID_ARG;
  if (max_len > 0x7fffffffLL) return DA_ERR_UNSUPPORTED;
  if (B == 0) return DA_OK;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(seq_lens, 4)) return DA_ERR_INVALID_ARG;
  const int rows = H * q_len, N = latent_tile_rows(rows), W = R + 64;
  if (max_len == 0 || (paged && num_pages == 0)) {
    if (cudaMemsetAsync(out, 0, (size_t)B * rows * R * 2, st) != cudaSuccess) {
      cudaGetLastError();
      return DA_ERR_CUDA;
    }
    return DA_OK;
  }
  if (!cache || !aligned(cache, 16)) return DA_ERR_INVALID_ARG;
  const int limit = R == 128 ? latent_batch_limit<128>(N) : R == 256 ? latent_batch_limit<256>(N)
                                                                     : latent_batch_limit<512>(N);
  if (B > limit) return DA_ERR_UNSUPPORTED;
  {
    // what is written overlaps nothing else of the call
    const long long qn = product(B, rows, W, 2), on = product(B, rows, R, 2);
    const long long cn = paged ? product(num_pages, page_size, W, 2) : product(B, max_len, W, 2);
    if (overlap(out, on, q, qn) || overlap(out, on, cache, cn) || overlap(out, on, workspace, workspace_bytes) ||
        overlap(workspace, workspace_bytes, q, qn) || overlap(workspace, workspace_bytes, cache, cn))
      return DA_ERR_INVALID_ARG;
  }
  int dev, sms, optin;
  if (current_device(&dev) || device_info(dev, &sms, &optin)) return DA_ERR_CUDA;
  if (!workspace || workspace_bytes < latent_workspace(B, rows, R, sms)) return DA_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return DA_ERR_INVALID_ARG;

  LatentParams prm;
  std::memset(&prm, 0, sizeof(prm));
  prm.U = (rows + N - 1) / N;
  // the plan counts line positions in 32 bits
  if ((long long)B * prm.U * ((max_len + kBlockTokens - 1) / kBlockTokens + 3 + kLatentGap) >= (1LL << 30))
    return DA_ERR_UNSUPPORTED;
  {
    const cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)(W / 64), (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)W * 2, 128, (cuuint64_t)rows * W * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)N, (cuuint32_t)(W / 64), 1};
    if (int e = encode_map_t(&prm.tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, q, 4, dims,
                             strides, box))
      return e;
  }
  // boxes of R rows of one page, the largest of 64, 32 and 16 that divides it; a box of two
  // columns has them 64 tokens apart only where it has all 64
  const int box_shift = !paged || page_size % 64 == 0 ? 2 : page_size % 32 == 0 ? 1 : 0;
  {
    const cuuint64_t slab = (cuuint64_t)(paged ? page_size : max_len);
    const cuuint64_t dims[4] = {64, slab, (cuuint64_t)(W / 64), (cuuint64_t)(paged ? num_pages : B)};
    const cuuint64_t strides[3] = {(cuuint64_t)W * 2, 128, slab * W * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)(16 << box_shift), (cuuint32_t)(box_shift == 2 ? 2 : 1), 1};
    const cuuint32_t box1[4] = {64, (cuuint32_t)(16 << box_shift), 1, 1};
    if (int e = encode_map_t(&prm.tm_unit, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, cache, 4,
                             dims, strides, box))
      return e;
    if (int e = encode_map_t(&prm.tm_pe, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, cache, 4, dims,
                             strides, box1))
      return e;
  }
  prm.seq_lens = seq_lens;
  prm.page_table = page_table;
  prm.part_acc = static_cast<float*>(workspace);
  prm.part_ml = reinterpret_cast<float2*>(prm.part_acc + latent_part_rows(rows, sms) * R);
  prm.pieces = reinterpret_cast<int4*>(prm.part_ml + latent_part_rows(rows, sms));
  prm.out = static_cast<__nv_bfloat16*>(out);
  prm.B = B;
  prm.H = H;
  prm.q_len = q_len;
  prm.rows = rows;
  prm.ranges = sms;
  prm.max_len = (int)max_len;
  prm.page_size = page_size;
  prm.max_pages = max_pages;
  prm.num_pages = num_pages;
  prm.box_shift = box_shift;
  prm.page_shift = paged && (page_size & (page_size - 1)) == 0 ? __builtin_ctz((unsigned)page_size) : -1;
  prm.scale_log2 = scale * kLog2e;
  prm.timeout_ns = kWaitTimeoutNs;
  switch (R) {
    case 128: return launch_latent_rows<128>(prm, N, paged, sms, dev, st);
    case 256: return launch_latent_rows<256>(prm, N, paged, sms, dev, st);
    default: return launch_latent_rows<512>(prm, N, paged, sms, dev, st);
  }
}

// CTAs a query block: where all CTAs of two parts a block still run at once, as many as do,
// up to the parts that the longest sequence there may be can have.  Blocks that see fewer
// keys have fewer parts, and their other CTAs leave at once (8 heads, 200 new tokens after
// 2800 keys: 22.4 us in a cache of that size and 24.2 in one of 131072; with parts sized by the
// capacity 52.0 there).  A second round of parts cost what the cut saved: 128 blocks of up to 21
// tiles (4 sequences, 16 heads, 500 new tokens) took 51.2 us whole and 47 to 54 in parts of 11
// to 8, by the sequences' order, before CTAs took over waiting blocks.
int prefill_parts(long long units, int max_ctx, int sms) {
  const int tiles = max_ctx / 128 + (max_ctx % 128 != 0);
  return units > 0 ? prefill_block_parts(tiles, (int)(sms / units)) : 1;
}

long long prefill_workspace(long long units, int max_ctx, int D, int sms) {
  const int parts = prefill_parts(units, max_ctx, sms);
  return parts == 1 ? 0 : units * parts * LatentPrefillGeo<128>::BQ * (D + 2) * 4;
}

template <int D>
int launch_latent_prefill(LatentPrefillParams& prm, const void* q, const void* k, const void* k_rope, const void* v,
                          long long token_stride, long long head_stride, long long rope_stride, int sms,
                          int dev, cudaStream_t st) {
  using Gm = LatentPrefillGeo<D>;
  static bool done[kMaxDevices] = {false}, fits[kMaxDevices] = {false};
  if (int e = allow_smem(latent_prefill_kernel<D>, Gm::SMEM, done, dev)) return e;
  {
    // the softmax warpgroups raise their registers out of what the launch gave the CTA; a
    // build whose per-thread count is below the split would wait for ever, so it is refused
    std::lock_guard<std::mutex> lk(g_mu);
    if (!fits[dev]) {
      cudaFuncAttributes fa;
      if (cudaFuncGetAttributes(&fa, latent_prefill_kernel<D>) != cudaSuccess) {
        cudaGetLastError();
        return DA_ERR_CUDA;
      }
      if (fa.numRegs * Gm::NTHREADS < Gm::REG_POOL_NEEDED) return DA_ERR_UNSUPPORTED;
      fits[dev] = true;
    }
  }
  const cuuint64_t L = (cuuint64_t)prm.max_len, H = (cuuint64_t)prm.H, B = (cuuint64_t)prm.B;
  const cuuint64_t ts = (cuuint64_t)token_stride * 2, hs = (cuuint64_t)head_stride * 2;
  const cuuint64_t dims[5] = {64, L, D / 64, H, B}, strides[4] = {ts, 128, hs, ts * L};
  const cuuint32_t box_k[5] = {64, 128, 1, 1, 1}, box_v[5] = {64, (cuuint32_t)Gm::VKEYS, D / 64, 1, 1};
  const cuuint64_t dims_pe[3] = {64, L, B}, strides_pe[2] = {(cuuint64_t)rope_stride * 2, (cuuint64_t)rope_stride * 2 * L};
  const cuuint32_t box_pe[3] = {64, 128, 1};
  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const cuuint64_t qw = Gm::W * 2;
  const cuuint64_t dims_q[5] = {64, (cuuint64_t)prm.q_len, Gm::W / 64, H, B};
  const cuuint64_t strides_q[4] = {qw * H, 128, qw, qw * H * (cuuint64_t)prm.q_len};
  const cuuint32_t box_q[5] = {64, Gm::M, Gm::W / 64, 1, 1};
  if (int e = encode_map_t(&prm.tm_q, bf16, sw, q, 5, dims_q, strides_q, box_q)) return e;
  if (int e = encode_map_t(&prm.tm_k, bf16, sw, k, 5, dims, strides, box_k)) return e;
  if (int e = encode_map_t(&prm.tm_v, bf16, sw, v, 5, dims, strides, box_v)) return e;
  if (int e = encode_map_t(&prm.tm_pe, bf16, sw, k_rope, 3, dims_pe, strides_pe, box_pe)) return e;
  {
    // launch groups of (b, h) units whose K/V fit in L2 together: the longest query blocks of
    // a group start first, so a second group's would start last (32 heads x 4096 tokens: 160 us
    // in groups of 24, 142 in one).  Where the capacity would make several groups, the kernel
    // takes the longest sequence's tokens instead (that prompt in a cache of 131072: 126 us, 157
    // in groups by the capacity; in a cache of its own size 124)
    const long long units = (long long)prm.B * prm.H;
    prm.grp = prefill_group(prm.max_len, D, units);
    prm.grp_by_length = prm.seq_lens && prm.grp < units;
  }
  const long long units = (long long)prm.nqb * prm.B * prm.H;
  if (units * prm.parts > 0x7fffffffLL) return DA_ERR_UNSUPPORTED;
  prm.more = units * prm.parts > sms;  // one CTA an SM
  if (int e = launch_dependent(latent_prefill_kernel<D>, (unsigned)(units * prm.parts), Gm::NTHREADS,
                               (size_t)Gm::SMEM, st, prm))
    return e;
  if (prm.parts == 1) return DA_OK;
  return launch_dependent(latent_prefill_merge<D>, (unsigned)(units * (Gm::BQ / 32)), 256, 0, st, prm);
}

}  // namespace
}  // namespace da

using namespace da;

extern "C" long long latent_workspace_bytes(int batch, int q_len, int num_heads, int latent_dim, int num_sms) {
  if (int e = latent_shape(batch, q_len, num_heads, latent_dim)) return -e;
  int dev, sms = num_sms, optin;
  if (sms <= 0 && (current_device(&dev) || device_info(dev, &sms, &optin))) return -DA_ERR_CUDA;
  return latent_workspace(batch, num_heads * q_len, latent_dim, sms);
}

extern "C" int latent_max_batch(int q_len, int num_heads, int latent_dim) {
  if (int e = latent_shape(1, q_len, num_heads, latent_dim)) return -e;
  const int N = latent_tile_rows(num_heads * q_len);
  return latent_dim == 128 ? latent_batch_limit<128>(N) : latent_dim == 256 ? latent_batch_limit<256>(N)
                                                                            : latent_batch_limit<512>(N);
}

extern "C" int latent_attn_contig(const void* q, const void* cache, const int* seq_lens, int batch, int q_len,
                                  int num_heads, int latent_dim, int max_ctx, float scale, void* workspace,
                                  long long workspace_bytes, void* out, void* stream) {
  if (max_ctx < 0) return DA_ERR_INVALID_ARG;
  return latent_call(false, q, cache, nullptr, seq_lens, batch, q_len, num_heads, latent_dim, max_ctx, 0, 0, 0, scale,
                     workspace, workspace_bytes, out, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int latent_attn_paged(const void* q, const void* pool, const int* page_table, const int* seq_lens,
                                 int batch, int q_len, int num_heads, int latent_dim, int page_size,
                                 int max_pages_per_seq, int num_pages, int max_seq_len, float scale, void* workspace,
                                 long long workspace_bytes, void* out, void* stream) {
  if (page_size <= 0 || max_pages_per_seq < 0 || num_pages < 0 || max_seq_len < 0) return DA_ERR_INVALID_ARG;
  if (page_size % 16 != 0) return DA_ERR_UNSUPPORTED;
  if (batch > 0 && (!seq_lens || !page_table || !aligned(page_table, 4))) return DA_ERR_INVALID_ARG;
  long long cap = (long long)max_pages_per_seq * page_size;
  if (cap > max_seq_len) cap = max_seq_len;
  return latent_call(true, q, pool, page_table, seq_lens, batch, q_len, num_heads, latent_dim, cap, page_size,
                     max_pages_per_seq, num_pages, scale, workspace, workspace_bytes, out,
                     reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int latent_prefill_contig(const void* q, const void* k_nope, const void* k_rope, const void* v,
                                     const int* seq_lens, int batch, int q_len, int num_heads, int head_dim,
                                     int max_ctx, long long kv_token_stride, long long kv_head_stride,
                                     long long rope_token_stride, float scale, void* workspace,
                                     long long workspace_bytes, void* out, void* stream) {
  if (batch < 0 || q_len < 0 || num_heads < 1 || max_ctx < 0 || !std::isfinite(scale)) return DA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return DA_ERR_UNSUPPORTED;
  if (batch == 0 || q_len == 0) return DA_OK;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(seq_lens, 4) || !aligned(workspace, 16))
    return DA_ERR_INVALID_ARG;
  const int BQ = LatentPrefillGeo<128>::BQ;
  const long long nqb = ((long long)q_len + BQ - 1) / BQ;
  if (nqb * batch > 0x7fffffffLL / num_heads) return DA_ERR_UNSUPPORTED;
  if (max_ctx > 0x7fffffff - BQ) return DA_ERR_UNSUPPORTED;  // a token past the last tile still counts in 32 bits
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (max_ctx == 0) {
    if (cudaMemsetAsync(out, 0, (size_t)batch * q_len * num_heads * head_dim * 2, st) != cudaSuccess) {
      cudaGetLastError();
      return DA_ERR_CUDA;
    }
    return DA_OK;
  }
  if (!k_nope || !k_rope || !v || !aligned(k_nope, 16) || !aligned(k_rope, 16) || !aligned(v, 16))
    return DA_ERR_INVALID_ARG;
  const long long far = 1LL << 40, cached = (long long)batch * max_ctx;
  if (kv_head_stride > far || kv_token_stride > far || rope_token_stride > far ||
      !reachable(num_heads, kv_head_stride) || !reachable(cached, kv_token_stride) ||
      !reachable(cached, rope_token_stride))
    return DA_ERR_INVALID_ARG;
  if (kv_head_stride < head_dim || kv_head_stride % 8 || kv_token_stride % 8 ||
      kv_token_stride < (num_heads - 1) * kv_head_stride + head_dim || rope_token_stride < 64 || rope_token_stride % 8)
    return DA_ERR_INVALID_ARG;
  {
    const long long on = product(batch, q_len, num_heads, head_dim, 2),
                    qn = product(batch, q_len, num_heads, head_dim + 64, 2);
    const long long tokens = cached - 1;
    const long long kn = (tokens * kv_token_stride + (num_heads - 1) * kv_head_stride + head_dim) * 2;
    const void* in[4] = {q, k_nope, v, k_rope};
    const long long bytes[4] = {qn, kn, kn, (tokens * rope_token_stride + 64) * 2};
    for (int i = 0; i < 4; ++i)
      if (overlap(out, on, in[i], bytes[i]) || overlap(workspace, workspace_bytes, in[i], bytes[i]))
        return DA_ERR_INVALID_ARG;
    if (overlap(out, on, workspace, workspace_bytes)) return DA_ERR_INVALID_ARG;
  }
  int dev, sms, optin;
  if (current_device(&dev) || device_info(dev, &sms, &optin)) return DA_ERR_CUDA;
  LatentPrefillParams prm;
  std::memset(&prm, 0, sizeof(prm));
  prm.out = static_cast<__nv_bfloat16*>(out);
  prm.seq_lens = seq_lens;
  prm.B = batch;
  prm.q_len = q_len;
  prm.H = num_heads;
  prm.nqb = (int)nqb;
  prm.max_len = max_ctx;
  prm.scale_log2 = scale * kLog2e;
  prm.timeout_ns = kWaitTimeoutNs;
  const long long units = nqb * batch * num_heads;
  prm.parts = 1;
  if (workspace) {
    if (workspace_bytes < prefill_workspace(units, max_ctx, head_dim, sms)) return DA_ERR_WORKSPACE;
    prm.parts = prefill_parts(units, max_ctx, sms);
    prm.part_acc = static_cast<float*>(workspace);
    prm.part_ml = reinterpret_cast<float2*>(prm.part_acc + units * prm.parts * BQ * head_dim);
  }
  return head_dim == 64 ? launch_latent_prefill<64>(prm, q, k_nope, k_rope, v, kv_token_stride, kv_head_stride,
                                                    rope_token_stride, sms, dev, st)
                        : launch_latent_prefill<128>(prm, q, k_nope, k_rope, v, kv_token_stride, kv_head_stride,
                                                     rope_token_stride, sms, dev, st);
}

extern "C" long long latent_prefill_workspace_bytes(int batch, int q_len, int num_heads, int head_dim, int max_ctx,
                                                    int num_sms) {
  if (batch < 0 || q_len < 0 || num_heads < 1 || max_ctx < 0) return -DA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return -DA_ERR_UNSUPPORTED;
  int dev, sms = num_sms, optin;
  if (sms <= 0 && (current_device(&dev) || device_info(dev, &sms, &optin))) return -DA_ERR_CUDA;
  const int BQ = LatentPrefillGeo<128>::BQ;
  const long long nqb = ((long long)q_len + BQ - 1) / BQ;
  if (nqb * batch > 0x7fffffffLL / num_heads) return -DA_ERR_UNSUPPORTED;
  return prefill_workspace(nqb * batch * num_heads, max_ctx, head_dim, sms);
}
