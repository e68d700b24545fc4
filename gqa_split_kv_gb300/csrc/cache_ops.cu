// Entry points around the caches (declared in include/decode_attn.h): rotary
// positions, writing new tokens into a cache (bf16 or quantised to int8) and reading a
// cache back as contiguous bf16.  All three move bytes: HBM (or, for a decode step's
// few tokens, the launch) bounds them, so every kernel is one pass with 16-byte
// accesses and the arithmetic between the load and the store.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/decode_attn.h"
#include "device_error.cuh"
#include "host_util.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace da {

int take_cache_error_word(unsigned int* flags) { return take_unit_error_word(flags); }

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRot = 2048;       // rotated elements of a head (cosines and sines sit in shared memory)
constexpr int kRopeSmem = 32 * 1024;

// ---------------------------------------------------------------- rope_apply

struct RopeApplyParams {
  RopeParams r;
  const void* x;
  void* out;
  const int* positions;
  long long tokens;
  int H, D;
  long long xt, xh, ot, oh;  // strides in elements
  int copy;                  // out is not x: elements outside the rotated part are copied
  int tb;                    // tokens a CTA takes at a time
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }

// A 16-byte chunk to and from fp32, two 16-bit elements an instruction.
template <typename T>
struct Chunk;
template <>
struct Chunk<float> {
  static __device__ __forceinline__ void unpack(uint4 w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct Chunk<__nv_bfloat16> {
  static __device__ __forceinline__ void unpack(uint4 w, float (&f)[8]) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16lo_to_f32(q[i]);
      f[2 * i + 1] = bf16hi_to_f32(q[i]);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Chunk<__half> {
  static __device__ __forceinline__ void unpack(uint4 w, float (&f)[8]) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = f16lo_to_f32(q[i]);
      f[2 * i + 1] = f16hi_to_f32(q[i]);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]),
                      pack_f16x2(f[6], f[7]));
  }
};

// The cosines and sines of pairs j .. j + n - 1 (j even: two pairs a read).
template <int N>
__device__ __forceinline__ void load_cs(const float2* cs, int j, float2 (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float4 c = *reinterpret_cast<const float4*>(cs + j + i);
    w[i] = make_float2(c.x, c.y);
    w[i + 1] = make_float2(c.z, c.w);
  }
}

// Rotates the pairs (a[i], b[i]), or the pairs of neighbours in a.
template <int V>
__device__ __forceinline__ void rotate_half(float (&a)[V], float (&b)[V], const float2* cs, int j) {
  float2 w[V];
  load_cs(cs, j, w);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float f = a[i], g = b[i];
    a[i] = f * w[i].x - g * w[i].y;
    b[i] = f * w[i].y + g * w[i].x;
  }
}
template <int V>
__device__ __forceinline__ void rotate_neighbours(float (&a)[V], const float2* cs, int j) {
  float2 w[V / 2];
  load_cs(cs, j, w);
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    const float f = a[i], g = a[i + 1];
    a[i] = f * w[i / 2].x - g * w[i / 2].y;
    a[i + 1] = f * w[i / 2].y + g * w[i / 2].x;
  }
}

// A CTA takes one token at a time (MANY: tb tokens): their rot / 2 cosines and sines go
// to shared memory once and serve every head.  VECTOR: all offsets and strides are whole
// 16-byte chunks; an item is a chunk (interleaved: whole pairs; a copy) or the two chunks
// that hold the halves of the same pairs.  Otherwise an item is one pair or one copied element.
//
// Bound by HBM (read and write once).  A thread's loads of the first U items go out
// before the position is known: with them after the cosines, a token takes two memory
// latencies and the sines in a row (4096 tokens x 32 heads x 128 bf16, neighbours: 22.5 us, now
// 14.8; floor 10.0).  fp32 gradients of 8192 tokens x 24 heads x 256, 64 elements of each
// turned: 62.5 us, floor 60.1, 6.4 TB/s.  One token each of 64 sequences: 2.8 us, a launch.
template <typename T, bool VECTOR, bool MANY>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeApplyParams p) {
  extern __shared__ __align__(16) uint8_t rope_smem[];
  const int np = p.r.rot / 2;
  unsigned long long* step = reinterpret_cast<unsigned long long*>(rope_smem);
  float2* cs = reinterpret_cast<float2*>(step + (np + 1) / 2 * 2);  // 16-byte aligned
  pdl_launch_dependents();
  pdl_wait_primary();
  for (int j = threadIdx.x; j < np; j += kThreads) step[j] = rope_turn_step(p.r.inv_freq[j]);
  constexpr int V = VECTOR ? 16 / (int)sizeof(T) : 1;
  constexpr int U = 2;  // items a thread has in flight
  // items of one head: the rotated ones first, then the copies
  const int nrot = VECTOR && p.r.interleaved ? p.r.rot / V : np / V;
  const int ncopy = p.copy ? (p.D - p.r.rot) / V : 0;
  const int per_head = nrot + ncopy, items = (MANY ? p.tb : 1) * p.H * per_head;
  const int lo = p.r.offset / V;  // copied items before the rotated part
  // this thread's first item is the same every time; kThreads items on is (di, dh, dk) on
  const int ih0 = threadIdx.x / per_head, k0 = threadIdx.x - ih0 * per_head;
  const int dih = kThreads / per_head, dk = kThreads - dih * per_head;
  const int i0 = MANY ? ih0 / p.H : 0, h0 = ih0 - i0 * p.H;
  const int di = MANY ? dih / p.H : 0, dh = dih - di * p.H;
  const int ci0 = MANY ? threadIdx.x / np : 0, cj0 = threadIdx.x - ci0 * np;
  const int dci = MANY ? kThreads / np : 0, dcj = kThreads - dci * np;
  const int second = VECTOR || !p.r.interleaved ? np : 1;  // from a pair's first half to its second
  const bool two = !(VECTOR && p.r.interleaved);           // the halves are loaded apart
  // an item's element (of the first of its two chunks or elements)
  auto place = [&](int k) {
    if (k < nrot) return VECTOR || !p.r.interleaved ? p.r.offset + k * V : p.r.offset + 2 * k;
    const int c = k - nrot;
    return (c < lo ? c : c + p.r.rot / V) * V;
  };
  using Item = typename std::conditional<VECTOR, uint4, T>::type;
  const int tb = MANY ? p.tb : 1;
  for (long long t0 = (long long)blockIdx.x * tb; t0 < p.tokens; t0 += (long long)gridDim.x * tb) {
    const int n = MANY ? (int)min((long long)tb, p.tokens - t0) : 1;
    const int pos = MANY ? 0 : load_dependent(p.positions + t0);
    const T* x = static_cast<const T*>(p.x) + t0 * p.xt;
    T* out = static_cast<T*>(p.out) + t0 * p.ot;
    int i = i0, h = h0, k = k0;
    for (int e0 = 0; e0 < items; e0 += U * kThreads) {
      Item a[U], b[U];
      int at[U], ti[U];
      bool rotates[U];
      long long oh[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool there = MANY ? i < n : h < p.H;
        rotates[u] = k < nrot && there;
        at[u] = there ? place(k) : -1;
        oh[u] = (MANY ? i * p.ot : 0) + h * p.oh;
        ti[u] = i;
        if (there) {
          const T* src = x + (MANY ? i * p.xt : 0) + h * p.xh + at[u];
          a[u] = *reinterpret_cast<const Item*>(src);
          if (rotates[u] && two) b[u] = *reinterpret_cast<const Item*>(src + second);
        }
        k += dk;
        h += dh;
        i += di;
        if (k >= per_head) {
          k -= per_head;
          ++h;
        }
        if (MANY && h >= p.H) {
          h -= p.H;
          ++i;
        }
      }
      if (e0 == 0) {      // the tokens' cosines
        __syncthreads();  // step is written; the last tokens' cosines are read
        if constexpr (MANY) {
          for (int c = ci0, j = cj0; c < n; c += dci, j += dcj) {
            if (j >= np) {
              j -= np;
              if (++c >= n) break;
            }
            cs[c * np + j] = rope_cos_sin(step[j], load_dependent(p.positions + t0 + c), p.r);
          }
        } else {
          for (int j = threadIdx.x; j < np; j += kThreads) cs[j] = rope_cos_sin(step[j], pos, p.r);
        }
        __syncthreads();
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (at[u] < 0) continue;
        T* o = out + oh[u] + at[u];
        if (rotates[u]) {
          if constexpr (VECTOR) {
            const int j = at[u] - p.r.offset;
            const float2* w = cs + (MANY ? ti[u] * np : 0);
            float f[V], g[V];
            Chunk<T>::unpack(a[u], f);
            if (two) {
              Chunk<T>::unpack(b[u], g);
              rotate_half(f, g, w, j);
              b[u] = Chunk<T>::pack(g);
            } else {
              rotate_neighbours(f, w, j / 2);
            }
            a[u] = Chunk<T>::pack(f);
          } else {
            const float2 w = cs[(MANY ? ti[u] * np : 0) + (p.r.interleaved ? (at[u] - p.r.offset) / 2 : at[u] - p.r.offset)];
            const float f = to_f32(a[u]), g = to_f32(b[u]);
            a[u] = from_f32<T>(f * w.x - g * w.y);
            b[u] = from_f32<T>(f * w.y + g * w.x);
          }
          if (two) *reinterpret_cast<Item*>(o + second) = b[u];
        }
        *reinterpret_cast<Item*>(o) = a[u];
      }
    }
  }
}

template <typename T>
int launch_rope(RopeApplyParams& p, int sms, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  const int half = p.r.interleaved ? p.r.rot : p.r.rot / 2;
  const bool vec = aligned(p.x, 16) && aligned(p.out, 16) && p.D % V == 0 && p.r.offset % V == 0 && half % V == 0 &&
                   p.r.rot % V == 0 && p.xt % V == 0 && p.xh % V == 0 && p.ot % V == 0 && p.oh % V == 0;
  // As many tokens as give every thread its U items, while there are 4 CTAs an SM (32768
  // tokens of one head of 64: 7.6 us, one at a time 36.6; 8 heads of 128: 29.5 and 55.2; one
  // token's work is faster without the divisions and registers of several: 32 heads of 128
  // neighbours, 4096 tokens, 14.8 us against 17.4)
  const int np = p.r.rot / 2, v = vec ? V : 1;
  const int items = p.H * ((vec && p.r.interleaved ? p.r.rot / v : np / v) + (p.copy ? (p.D - p.r.rot) / v : 0));
  const long long room = kRopeSmem / (8 * np) - 2, even = p.tokens / (4 * sms);
  long long tb = 2 * kThreads / items;
  tb = tb > even ? even : tb;
  tb = tb > room ? room : tb;
  p.tb = tb < 1 ? 1 : (int)tb;
  const size_t smem = (size_t)((np + 1) / 2 * 2 + p.tb * np) * 8;
  // CTAs that go through several tokens: 16 an SM, 5 to 8 of them at once (the gradients above: 62.5
  // us, 68.3 with 8)
  const long long cap = (p.tb > 1 ? 8LL : 16LL) * sms, blocks = (p.tokens + p.tb - 1) / p.tb;
  const unsigned grid = (unsigned)(blocks < cap ? blocks : cap);
  if (p.tb > 1)
    return vec ? launch_dependent(rope_kernel<T, true, true>, grid, kThreads, smem, st, p)
               : launch_dependent(rope_kernel<T, false, true>, grid, kThreads, smem, st, p);
  return vec ? launch_dependent(rope_kernel<T, true, false>, grid, kThreads, smem, st, p)
             : launch_dependent(rope_kernel<T, false, false>, grid, kThreads, smem, st, p);
}

int rope_check(const double* inv_freq, int head_dim, int offset, int rot, int interleaved, float magnitude) {
  if (!inv_freq || !aligned(inv_freq, 8) || rot < 2 || rot % 2 || offset < 0 || (long long)offset + rot > head_dim ||
      (interleaved != 0 && interleaved != 1) || !std::isfinite(magnitude))
    return DA_ERR_INVALID_ARG;
  return rot > kMaxRot ? DA_ERR_UNSUPPORTED : DA_OK;
}

// [T, H, D] with these strides: whether two (token, head) rows can share an element.
bool rows_apart(long long T, long long H, long long D, long long st, long long sh) {
  if (T <= 1) st = 0;
  if (H <= 1) sh = 0;
  const bool th = (H <= 1 || sh >= D) && (T <= 1 || st >= (H - 1) * sh + D);
  const bool ht = (T <= 1 || st >= D) && (H <= 1 || sh >= (T - 1) * st + D);
  return th || ht;
}

// ---------------------------------------------------------------- the caches

struct CacheParams {
  RopeParams r;
  const void *k_new, *v_new;  // write: the new tokens; read: the outputs
  void *k_out, *v_out;
  void *k, *v;                // the cache
  float *ks, *vs;             // int8: its scales, [B or pages, Hkv, max_ctx or page_size]
  const int *seq_lens, *starts, *page_table;
  long long k_stride, v_stride;  // write: elements between new tokens
  int B, n, Hkv, D;           // n: tokens a sequence of this call
  int cap;                    // tokens a sequence has room for
  int slab;                   // rows of one batch entry or page: max_ctx or page_size
  int max_pages, num_pages;
  int tb;                     // tokens a CTA takes at a time
  int lanes;                  // write: lanes a row (a power of two)
  int fill;                   // read: rows with no token are written, as zeros
};

// The cache row (in tokens) of sequence b's position t, or -1 when its page is not in
// the pool (flagged); slab_index and in_slab address its scale.
template <bool PAGED>
__device__ __forceinline__ long long cache_row(const CacheParams& p, int b, int t, long long& slab_index,
                                               int& in_slab) {
  if (!PAGED) {
    slab_index = b;
    in_slab = t;
  } else {
    const int col = t / p.slab;
    const int page = load_dependent(p.page_table + (size_t)b * p.max_pages + col);
    if ((unsigned)page >= (unsigned)p.num_pages) {
      atomicOr(&g_error_word, 4u);
      return -1;
    }
    slab_index = page;
    in_slab = t - col * p.slab;
  }
  return slab_index * p.slab + in_slab;
}

// The larger one; NaN when either is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// A CTA takes tb new tokens at a time.  A row (token, tensor, head) of D elements has
// `lanes` lanes of one warp, CPL chunks of 8 elements each.  K rows are rotated in fp32
// on the way (a half-layout lane also loads the chunk with the other halves of its
// pairs: an L1 hit) and int8 rows quantised from that fp32 value, so a key is rounded
// once.  The row's maximum is a shuffle over its lanes.  Bound by HBM for a chunk and by
// latency for a step: the first rows' loads go out before the lengths, pages and cosines,
// which are looked up once a token.  A decode step of 64 sequences (8 heads x 128, int8 pages)
// with its read back: 6.0 us, two launches; 4096 tokens likewise 20.2 us, floor 7.6; 32768
// tokens 53.0 us here, floor 30.4 (bf16 48.0, 40.1), where four-chunk rows take 22 instructions
// an element and one-chunk rows took 31.
constexpr int kMaxTokens = 16;  // tokens a CTA takes at a time, at most
template <bool PAGED, bool INT8, int CPL, bool PAIRED>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const CacheParams p) {
  extern __shared__ __align__(16) uint8_t rope_smem[];
  // where a token's first head begins in the cache, or -1; its first head's scale
  __shared__ long long tok_at[kMaxTokens], tok_scale[kMaxTokens];
  const int np = p.r.inv_freq ? p.r.rot / 2 : 0;
  unsigned long long* step = reinterpret_cast<unsigned long long*>(rope_smem);
  float2* cs = reinterpret_cast<float2*>(step + np);  // [tb][np] (np a multiple of 8)
  const unsigned total = (unsigned)p.B * (unsigned)p.n;  // below 2^31
  const int rows_per_token = p.Hkv * (p.v_new ? 2 : 1);
  const int rows = p.tb * rows_per_token;
  const int nchunk = p.D / 8, gl = threadIdx.x & (p.lanes - 1);
  // position of new token g = b n + i: L_b - n + i
  auto position = [&](unsigned g, int& b) -> long long {
    b = (int)(g / (unsigned)p.n);
    const int L = p.seq_lens ? load_dependent(p.seq_lens + b) : p.cap;
    return (long long)L - p.n + (int)(g - (unsigned)b * (unsigned)p.n);
  };
  pdl_launch_dependents();
  pdl_wait_primary();
  bool first = true;
  // every lane of a warp runs the same number of rounds (the shuffles need them all); a
  // thread's rows and cosines are the same of every tb tokens, and the next ones a fixed step on
  const int per_round = kThreads / p.lanes;
  const int row0 = threadIdx.x / p.lanes, ti0 = row0 / rows_per_token, in0 = row0 - ti0 * rows_per_token;
  const int dti = per_round / rows_per_token, din = per_round - dti * rows_per_token;
  const int ci0 = np ? threadIdx.x / np : 0, cj0 = threadIdx.x - ci0 * np;
  const int dci = np ? kThreads / np : 0, dcj = kThreads - dci * np;
  for (unsigned g0 = blockIdx.x * p.tb; g0 < total; g0 += gridDim.x * p.tb) {
    int ti = ti0, in_token = in0;
    for (int r0 = 0; r0 < rows; r0 += per_round, ti += dti, in_token += din) {
      if (in_token >= rows_per_token) {
        in_token -= rows_per_token;
        ++ti;
      }
      const bool is_v = in_token >= p.Hkv;
      const int h = is_v ? in_token - p.Hkv : in_token;
      const unsigned g = g0 + ti;
      const bool there = ti < p.tb && g < total;
      // the row's elements do not depend on its place, so their loads go out first
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? p.v_new : p.k_new) +
                                 (there ? g * (is_v ? p.v_stride : p.k_stride) + h * p.D : 0);
      const bool rotates = np && !is_v;
      uint4 raw[CPL], other[CPL];
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const int ch = gl + c * p.lanes;
        raw[c] = other[c] = make_uint4(0u, 0u, 0u, 0u);
        if (there && ch < nchunk) {
          raw[c] = load_dependent(reinterpret_cast<const uint4*>(src) + ch);
          const int at = ch * 8 - p.r.offset;  // within the rotated part
          if (!PAIRED && rotates && !p.r.interleaved && at >= 0 && at < p.r.rot)  // the other halves of these pairs
            other[c] =
                load_dependent(reinterpret_cast<const uint4*>(src + p.r.offset + (at >= np ? at - np : at + np)));
        }
      }
      if (r0 == 0) {  // the tokens' places and cosines
        if (first)
          for (int j = threadIdx.x; j < np; j += kThreads) step[j] = rope_turn_step(p.r.inv_freq[j]);
        first = false;
        __syncthreads();  // step is written; the last tokens' cosines and places are read
        const int helper = (int)kThreads - 1 - (int)threadIdx.x;  // the last threads have the fewest cosines
        if (helper < p.tb) {
          long long slab = 0, place = -1;
          int in_slab = 0, b;
          if (g0 + helper < total) {
            const long long pos = position(g0 + helper, b);
            if (pos >= p.cap)
              atomicOr(&g_error_word, 8u);
            else if (pos >= 0)
              place = cache_row<PAGED>(p, b, (int)pos, slab, in_slab);
          }
          tok_at[helper] = place < 0 ? -1 : place * p.Hkv * p.D;
          tok_scale[helper] = slab * p.Hkv * p.slab + in_slab;
        }
        for (int i = ci0, j = cj0; i < p.tb && np; i += dci, j += dcj) {
          if (j >= np) {
            j -= np;
            if (++i >= p.tb) break;
          }
          int b;
          if (g0 + i < total) cs[i * np + j] = rope_cos_sin(step[j], (int)position(g0 + i, b), p.r);
        }
        __syncthreads();
      }
      const long long dst = there ? tok_at[ti] : -1;
      float x[CPL][8];
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        Chunk<__nv_bfloat16>::unpack(raw[c], x[c]);
        if (PAIRED) continue;
        const int at = (gl + c * p.lanes) * 8 - p.r.offset;
        if (rotates && there && at >= 0 && at < p.r.rot) {
          const float2* w = cs + ti * np;
          if (p.r.interleaved) {
            rotate_neighbours(x[c], w, at / 2);
          } else {
            float o[8];
            Chunk<__nv_bfloat16>::unpack(other[c], o);
            if (at >= np)
              rotate_half(o, x[c], w, at - np);
            else
              rotate_half(x[c], o, w, at);
          }
        }
      }
      if (PAIRED && rotates && there)
#pragma unroll
        for (int c = 0; c < CPL / 2; ++c)
          rotate_half(x[c], x[c + CPL / 2], cs + ti * np, (gl + c * p.lanes) * 8);
      if constexpr (INT8) {
        // The largest magnitude, then by its bits, whose order is that of the magnitudes, with
        // infinity and the NaNs above them: a row with any of those gets a NaN scale and zeros.
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < CPL; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) top = max_or_nan(top, fabsf(x[c][i]));
        unsigned bits = __float_as_uint(top) & 0x7fffffffu;
        for (int o = p.lanes / 2; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
        const bool finite = bits < 0x7f800000u;
        top = __uint_as_float(bits);
        // 127 2^-126 and less would leave a scale below the normal numbers: floor it
        float scale = bits ? fmaxf(__fdiv_rn(top, 127.f), 1.17549435e-38f) : 1.f;
        // x / scale, rounded as a division is: a quotient from the rounded reciprocal and one
        // correction by its remainder (Markstein); adding 1.5 2^23 leaves the nearest integer,
        // ties to even, in the low bits, and no quotient passes 127 by half a step
        const float inv = __frcp_rn(scale);
        if (!finite) scale = __int_as_float(0x7fffffff);
        if (dst >= 0) {
          int8_t* q = static_cast<int8_t*>(is_v ? p.v : p.k) + dst + h * p.D;
#pragma unroll
          for (int c = 0; c < CPL; ++c) {
            const int ch = gl + c * p.lanes;
            if (ch >= nchunk) continue;
            uint32_t n[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float r = x[c][i] * inv;
              n[i] = __float_as_uint(fmaf(fmaf(-r, scale, x[c][i]), inv, r) + 12582912.f);
            }
            uint2 w;
            w.x = __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
            w.y = __byte_perm(__byte_perm(n[4], n[5], 0x0040), __byte_perm(n[6], n[7], 0x0040), 0x5410);
            if (!finite) w = make_uint2(0u, 0u);
            *reinterpret_cast<uint2*>(q + ch * 8) = w;
          }
          if (gl == 0) (is_v ? p.vs : p.ks)[tok_scale[ti] + (long long)h * p.slab] = scale;
        }
      } else if (dst >= 0) {
        __nv_bfloat16* q = static_cast<__nv_bfloat16*>(is_v ? p.v : p.k) + dst + h * p.D;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
          const int ch = gl + c * p.lanes;
          if (ch < nchunk) *reinterpret_cast<uint4*>(q + ch * 8) = rotates ? Chunk<__nv_bfloat16>::pack(x[c]) : raw[c];
        }
      }
    }
  }
}

// A CTA reads tb consecutive tokens of one sequence, 16 bytes of the cache a thread and
// step (int8: 32 bytes written).  FILL: rows with no token are written too, as zeros.  Bound
// by HBM: 16 ragged sequences up to 8192 tokens, 8 heads x 128 from int8 pages, 72.8 us, floor
// 62.6 (5.8 TB/s), and filled 109.4 us, floor 102.5; one sequence of 4096 tokens, 4 heads x
// 256: 6.0 us, floor 3.8.  The warps in flight hide the chain page, row, store: with two
// items a thread the batch takes 84 us, with both tensors' loads before the first store 78.6.
template <bool PAGED, bool INT8, bool FILL>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const CacheParams p) {
  const int nblk = (int)(((long long)p.n + p.tb - 1) / p.tb);
  const int b = blockIdx.x / nblk, i0 = (blockIdx.x - b * nblk) * p.tb;
  pdl_launch_dependents();
  pdl_wait_primary();
  int L = p.seq_lens ? load_dependent(p.seq_lens + b) : p.cap;
  L = min(L, p.cap);
  const int start = p.starts ? load_dependent(p.starts + b) : 0;
  constexpr int E = INT8 ? 16 : 8;  // elements of a 16-byte load
  const int per_row = p.Hkv * p.D / E, per_head = p.D / E;
  const int ntok = min(p.tb, p.n - i0);
  const int tensors = p.v_out ? 2 : 1;
  for (int e = threadIdx.x; e < ntok * per_row; e += kThreads) {
    const int ti = e / per_row, c = e - ti * per_row;
    const long long t = (long long)start + i0 + ti;
    long long slab, row = -1;
    int in_slab;
    if (t >= 0 && t < L) row = cache_row<PAGED>(p, b, (int)t, slab, in_slab);
    const size_t dst = ((size_t)b * p.n + i0 + ti) * per_row + c;
    if (row < 0) {
      if (!FILL) continue;
      for (int kv = 0; kv < tensors; ++kv) {
        uint4* out = reinterpret_cast<uint4*>(kv ? p.v_out : p.k_out) + (INT8 ? 2 : 1) * dst;
        out[0] = make_uint4(0u, 0u, 0u, 0u);
        if (INT8) out[1] = make_uint4(0u, 0u, 0u, 0u);
      }
      continue;
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      if (kv >= tensors) break;
      uint4* out = reinterpret_cast<uint4*>(kv ? p.v_out : p.k_out) + (INT8 ? 2 : 1) * dst;
      const uint4 w = load_dependent(reinterpret_cast<const uint4*>(kv ? p.v : p.k) + row * per_row + c);
      if constexpr (!INT8) {
        out[0] = w;
      } else {
        const float s = load_dependent((kv ? p.vs : p.ks) + (slab * p.Hkv + c / per_head) * p.slab + in_slab);
        const uint32_t q[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[2 * i] = pack_bf16x2((float)(int8_t)(q[i]) * s, (float)(int8_t)(q[i] >> 8) * s);
          o[2 * i + 1] = pack_bf16x2((float)(int8_t)(q[i] >> 16) * s, (float)(int8_t)(q[i] >> 24) * s);
        }
        out[0] = make_uint4(o[0], o[1], o[2], o[3]);
        out[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

int check_cache(const CacheParams& p, bool paged, bool int8, long long cap) {
  if (p.B < 0 || p.n < 0 || p.Hkv <= 0 || p.D <= 0 || cap < 0) return DA_ERR_INVALID_ARG;
  if (p.D % (int8 ? 16 : 8) || p.D > 1024 || p.Hkv > 1024 || cap > 0x7fffffffLL) return DA_ERR_UNSUPPORTED;
  if (paged && (p.slab <= 0 || p.max_pages < 0 || p.num_pages < 0)) return DA_ERR_INVALID_ARG;
  if ((long long)p.B * p.n > 0x7fffffffLL) return DA_ERR_UNSUPPORTED;
  return DA_OK;
}

// Bytes of one tensor of the cache, and of its scales.
long long cache_bytes(const CacheParams& p, bool paged, bool int8) {
  return product(paged ? p.num_pages : p.B, p.slab, p.Hkv, p.D, int8 ? 1 : 2);
}
long long scale_bytes(const CacheParams& p, bool paged) {
  return product(paged ? p.num_pages : p.B, p.slab, p.Hkv, 4);
}

int check_cache_pointers(const CacheParams& p, bool paged, bool int8, bool has_v) {
  const bool rows = p.cap > 0 && (!paged || p.num_pages > 0);  // a cache of none may be null
  if (rows && (!p.k || !p.v != !has_v)) return DA_ERR_INVALID_ARG;
  if (!aligned(p.k, 16) || !aligned(p.v, 16)) return DA_ERR_INVALID_ARG;
  if (int8 && rows && (!p.ks || (has_v && !p.vs))) return DA_ERR_INVALID_ARG;
  if (!aligned(p.ks, 4) || !aligned(p.vs, 4)) return DA_ERR_INVALID_ARG;
  if (paged && (!p.page_table || !p.seq_lens || !aligned(p.page_table, 4))) return DA_ERR_INVALID_ARG;
  if (!aligned(p.seq_lens, 4) || !aligned(p.starts, 4)) return DA_ERR_INVALID_ARG;
  return DA_OK;
}

template <bool PAGED, bool INT8>
int launch_write(CacheParams& p, int sms, cudaStream_t st) {
  // Few rows: a chunk a lane, for more loads at once.  Many (20 an SM): two chunks, and int8
  // four where the 16 tokens of a CTA still occupy it, as a row's fixed work is a lane's (8 heads x 128,
  // int8 / bf16, us: 128 tokens 3.2 / 2.9, 3.6 / 2.7 with more chunks; 256 tokens 4.4 / 3.4 -> 3.8 /
  // 2.9; 32768 tokens int8 56.0 with two, 53.0 with four, where bf16 takes 48.0 and 51.0)
  const int nchunk = p.D / 8;
  const int rows = p.Hkv * (p.v_new ? 2 : 1), np = p.r.inv_freq ? p.r.rot / 2 : 0;
  const bool many = (long long)p.B * p.n * rows >= 20LL * sms;
  int cpl = nchunk > 64 ? 4 : nchunk > 32 || (nchunk > 1 && many) ? 2 : 1;
  // no rotation, or pairs whose halves a lane with an even number of chunks holds both
  bool paired = np == 0 || (!p.r.interleaved && p.r.offset == 0 && p.r.rot == p.D);
  if (INT8 && paired && many && (nchunk == 16 || nchunk == 32) && rows * (nchunk / 4) * kMaxTokens >= kThreads) cpl = 4;
  p.lanes = 1;
  while (p.lanes * cpl < nchunk && p.lanes < 32) p.lanes *= 2;
  paired = paired && (cpl == 2 || (INT8 && cpl == 4)) && (np == 0 || p.lanes * cpl == nchunk);
  // enough tokens that every lane has a row, four rounds of them where tokens abound (the
  // cosines then take every thread), as long as the cosines fit
  const long long total = (long long)p.B * p.n;
  p.tb = kThreads / (rows * p.lanes);
  p.tb = p.tb < 1 ? 1 : p.tb;
  while (p.tb < 4 && total >= 12LL * sms * p.tb) p.tb *= 2;
  const int room = np ? kRopeSmem / (8 * np) - 1 : kMaxTokens;
  p.tb = p.tb > kMaxTokens ? kMaxTokens : p.tb;
  p.tb = p.tb > room ? room : p.tb;
  const long long blocks = (total + p.tb - 1) / p.tb, cap = 8LL * sms;
  const unsigned grid = (unsigned)(blocks < cap ? blocks : cap);
  const size_t smem = (size_t)np * 8 * (1 + p.tb);
  if constexpr (INT8)
    if (paired && cpl == 4) return launch_dependent(kv_write_kernel<PAGED, INT8, 4, true>, grid, kThreads, smem, st, p);
  if (paired) return launch_dependent(kv_write_kernel<PAGED, INT8, 2, true>, grid, kThreads, smem, st, p);
  if (cpl == 1) return launch_dependent(kv_write_kernel<PAGED, INT8, 1, false>, grid, kThreads, smem, st, p);
  if (cpl == 2) return launch_dependent(kv_write_kernel<PAGED, INT8, 2, false>, grid, kThreads, smem, st, p);
  return launch_dependent(kv_write_kernel<PAGED, INT8, 4, false>, grid, kThreads, smem, st, p);
}

int write_call(bool paged, bool int8, CacheParams& p, long long cap, cudaStream_t st) {
  if (int e = check_cache(p, paged, int8, cap)) return e;
  p.cap = (int)cap;
  if (p.r.inv_freq) {
    if (int e = rope_check(p.r.inv_freq, p.D, p.r.offset, p.r.rot, p.r.interleaved, p.r.magnitude)) return e;
    if (p.r.offset % 8 || p.r.rot % 16) return DA_ERR_UNSUPPORTED;  // whole chunks of 8, in either layout
  }
  if (p.B == 0 || p.n == 0) return DA_OK;
  const long long width = (long long)p.Hkv * p.D;
  const bool has_v = p.v_new != nullptr;
  if (!p.k_new || !aligned(p.k_new, 16) || !aligned(p.v_new, 16)) return DA_ERR_INVALID_ARG;
  const long long far = 1LL << 40, new_tokens = (long long)p.B * p.n;
  if (p.k_stride < width || p.k_stride % 8 || p.k_stride > far || !reachable(new_tokens, p.k_stride) ||
      (has_v && (p.v_stride < width || p.v_stride % 8 || p.v_stride > far || !reachable(new_tokens, p.v_stride))))
    return DA_ERR_INVALID_ARG;
  if (!has_v && p.v) return DA_ERR_INVALID_ARG;
  if (int e = check_cache_pointers(p, paged, int8, has_v)) return e;
  {
    // nothing that is written may be read by the same call, nor written twice
    const long long tokens = new_tokens - 1, kn = (tokens * p.k_stride + width) * 2,
                    vn = has_v ? (tokens * p.v_stride + width) * 2 : 0, cn = cache_bytes(p, paged, int8),
                    sn = scale_bytes(p, paged);
    const void* dst[4] = {p.k, p.v, p.ks, p.vs};
    const long long bytes[4] = {cn, cn, sn, sn};
    for (int i = 0; i < 4; ++i) {
      if (overlap(p.k_new, kn, dst[i], bytes[i]) || overlap(p.v_new, vn, dst[i], bytes[i])) return DA_ERR_INVALID_ARG;
      for (int j = 0; j < i; ++j)
        if (overlap(dst[j], bytes[j], dst[i], bytes[i])) return DA_ERR_INVALID_ARG;
    }
  }
  int dev, sms, optin;
  if (current_device(&dev) || device_info(dev, &sms, &optin)) return DA_ERR_CUDA;
  if (paged) return int8 ? launch_write<true, true>(p, sms, st) : launch_write<true, false>(p, sms, st);
  return int8 ? launch_write<false, true>(p, sms, st) : launch_write<false, false>(p, sms, st);
}

int read_call(bool paged, bool int8, CacheParams& p, long long cap, cudaStream_t st) {
  if (int e = check_cache(p, paged, int8, cap)) return e;
  p.cap = (int)cap;
  if (p.B == 0 || p.n == 0) return DA_OK;
  const bool has_v = p.v_out != nullptr;
  if (!p.k_out || !aligned(p.k_out, 16) || !aligned(p.v_out, 16) || (!has_v && p.v)) return DA_ERR_INVALID_ARG;
  if (int e = check_cache_pointers(p, paged, int8, has_v)) return e;
  if (p.cap == 0 || (paged && p.num_pages == 0)) {  // there is no token
    const size_t bytes = (size_t)p.B * p.n * p.Hkv * p.D * 2;
    if (p.fill && (cudaMemsetAsync(p.k_out, 0, bytes, st) != cudaSuccess ||
                   (has_v && cudaMemsetAsync(p.v_out, 0, bytes, st) != cudaSuccess))) {
      cudaGetLastError();
      return DA_ERR_CUDA;
    }
    return DA_OK;
  }
  {
    const long long on = product(p.B, p.n, p.Hkv, p.D, 2), cn = cache_bytes(p, paged, int8),
                    sn = scale_bytes(p, paged);
    const void *out[2] = {p.k_out, p.v_out}, *src[4] = {p.k, p.v, p.ks, p.vs};
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 4; ++j)
        if (overlap(out[i], on, src[j], j < 2 ? cn : sn)) return DA_ERR_INVALID_ARG;
    if (overlap(out[0], on, out[1], on)) return DA_ERR_INVALID_ARG;
  }
  int dev, sms, optin;
  if (current_device(&dev) || device_info(dev, &sms, &optin)) return DA_ERR_CUDA;
  // about 4 loads of 16 bytes a thread and tensor, fewer while that leaves SMs without their
  // 2048 threads (4096 tokens x 8 heads x 128 from int8: 11 us at 4, 256 CTAs)
  const int per_row = p.Hkv * p.D / (int8 ? 16 : 8);
  int tb = kThreads * 4 / per_row;
  tb = tb < 1 ? 1 : tb > 64 ? 64 : tb;
  auto blocks = [&](int t) { return p.B * (((long long)p.n + t - 1) / t); };
  while (tb > 1 && tb * per_row > kThreads && blocks(tb) < 8LL * sms) tb = (tb + 1) / 2;
  p.tb = tb;
  const long long grid = blocks(tb);
  if (grid > 0x7fffffffLL) return DA_ERR_UNSUPPORTED;
  auto launch = [&](auto in_pages, auto in_int8) {
    constexpr bool P = decltype(in_pages)::value, I = decltype(in_int8)::value;
    return p.fill ? launch_dependent(kv_read_kernel<P, I, true>, (unsigned)grid, kThreads, 0, st, p)
                  : launch_dependent(kv_read_kernel<P, I, false>, (unsigned)grid, kThreads, 0, st, p);
  };
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  return paged && int8 ? launch(yes, yes) : paged ? launch(yes, no) : launch(no, yes);
}

long long paged_cap(int page_size, int max_pages, int max_seq_len) {
  if (max_seq_len < 0 || page_size <= 0 || max_pages < 0) return -1;
  const long long room = (long long)max_pages * page_size;
  return room < max_seq_len ? room : max_seq_len;
}

}  // namespace
}  // namespace da

using namespace da;

extern "C" int rope_inv_freq(double* inv_freq, int rot_dim, double base, int scaling, double factor,
                             double original_ctx, double low_turns, double high_turns) {
  const double two_pi = 6.283185307179586476925;
  if (!inv_freq || rot_dim < 2 || rot_dim % 2 || !(base > 1.0) || !std::isfinite(base)) return DA_ERR_INVALID_ARG;
  if (scaling < DA_ROPE_PLAIN || scaling > DA_ROPE_BY_PARTS) return DA_ERR_UNSUPPORTED;
  if (scaling != DA_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return DA_ERR_INVALID_ARG;
  if (scaling == DA_ROPE_BASE && rot_dim == 2) return DA_ERR_INVALID_ARG;  // one pair, of frequency 1 under any base
  if (scaling == DA_ROPE_BY_PARTS && (!(original_ctx > 0) || !std::isfinite(original_ctx) || !(low_turns >= 0) ||
                                      !(high_turns > low_turns) || !std::isfinite(high_turns)))
    return DA_ERR_INVALID_ARG;
  if (scaling == DA_ROPE_BASE) base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
  for (int j = 0; j < rot_dim / 2; ++j) {
    double w = std::pow(base, -2.0 * j / rot_dim);
    if (scaling == DA_ROPE_LINEAR) w /= factor;
    if (scaling == DA_ROPE_BY_PARTS) {
      const double turns = original_ctx * w / two_pi;
      double keep = (turns - low_turns) / (high_turns - low_turns);
      keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      w = w * keep + w / factor * (1.0 - keep);
    }
    inv_freq[j] = w;
  }
  return DA_OK;
}

extern "C" int rope_apply(const void* x, void* out, const int* positions, const double* inv_freq, long long tokens,
                          int num_heads, int head_dim, int rot_offset, int rot_dim, int interleaved, float magnitude,
                          int backward, int dtype, long long x_token_stride, long long x_head_stride,
                          long long out_token_stride, long long out_head_stride, void* stream) {
  if (tokens < 0 || num_heads <= 0 || head_dim <= 0) return DA_ERR_INVALID_ARG;
  if (dtype < DA_BF16 || dtype > DA_F32) return DA_ERR_UNSUPPORTED;
  if (int e = rope_check(inv_freq, head_dim, rot_offset, rot_dim, interleaved, magnitude)) return e;
  if ((long long)num_heads * head_dim > 0x1fffffffLL) return DA_ERR_UNSUPPORTED;
  if (tokens == 0) return DA_OK;
  const int size = dtype == DA_F32 ? 4 : 2;
  if (!x || !out || !positions || !aligned(x, size) || !aligned(out, size) || !aligned(positions, 4))
    return DA_ERR_INVALID_ARG;
  const long long far = 1LL << 40;
  if (tokens > 0x7fffffffLL || x_token_stride > far || x_head_stride > far || out_token_stride > far ||
      out_head_stride > far || !reachable(tokens, x_token_stride) || !reachable(num_heads, x_head_stride) ||
      !reachable(tokens, out_token_stride) || !reachable(num_heads, out_head_stride))
    return DA_ERR_INVALID_ARG;
  if (!rows_apart(tokens, num_heads, head_dim, out_token_stride, out_head_stride)) return DA_ERR_INVALID_ARG;
  const bool same = x == out;
  if (same) {
    if ((tokens > 1 && x_token_stride != out_token_stride) || (num_heads > 1 && x_head_stride != out_head_stride))
      return DA_ERR_INVALID_ARG;
  } else {
    // a partly overlapping output would be read after it is written
    const long long xn = ((tokens - 1) * x_token_stride + (num_heads - 1) * x_head_stride + head_dim) * size;
    const long long on = ((tokens - 1) * out_token_stride + (num_heads - 1) * out_head_stride + head_dim) * size;
    if (overlap(x, xn, out, on)) return DA_ERR_INVALID_ARG;
  }
  int dev, sms, optin;
  if (current_device(&dev) || device_info(dev, &sms, &optin)) return DA_ERR_CUDA;
  RopeApplyParams p;
  p.r = {inv_freq, rot_offset, rot_dim, interleaved, magnitude, backward ? -1.f : 1.f};
  p.x = x;
  p.out = out;
  p.positions = positions;
  p.tokens = tokens;
  p.H = num_heads;
  p.D = head_dim;
  p.xt = x_token_stride;
  p.xh = x_head_stride;
  p.ot = out_token_stride;
  p.oh = out_head_stride;
  p.copy = !same;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == DA_BF16 ? launch_rope<__nv_bfloat16>(p, sms, st)
         : dtype == DA_F16 ? launch_rope<__half>(p, sms, st) : launch_rope<float>(p, sms, st);
}

namespace {

CacheParams write_params(const void* k_new, const void* v_new, long long k_stride, long long v_stride,
                         const int* seq_lens, int batch, int q_len, int num_kv_heads, int head_dim,
                         const double* inv_freq, int rot_offset, int rot_dim, int interleaved, float magnitude,
                         void* k, void* v, float* ks, float* vs) {
  CacheParams p = {};
  p.r = {inv_freq, rot_offset, rot_dim, interleaved, magnitude, 1.f};
  p.k_new = k_new;
  p.v_new = v_new;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.seq_lens = seq_lens;
  p.B = batch;
  p.n = q_len;
  p.Hkv = num_kv_heads;
  p.D = head_dim;
  p.k = k;
  p.v = v;
  p.ks = ks;
  p.vs = vs;
  return p;
}

CacheParams read_params(const void* k, const void* v, const float* ks, const float* vs, const int* starts,
                        const int* seq_lens, int batch, int n_tokens, int num_kv_heads, int head_dim, void* k_out,
                        void* v_out, bool fill) {
  CacheParams p = {};
  p.k = const_cast<void*>(k);
  p.v = const_cast<void*>(v);
  p.ks = const_cast<float*>(ks);
  p.vs = const_cast<float*>(vs);
  p.starts = starts;
  p.seq_lens = seq_lens;
  p.B = batch;
  p.n = n_tokens;
  p.Hkv = num_kv_heads;
  p.D = head_dim;
  p.k_out = k_out;
  p.v_out = v_out;
  p.fill = fill;
  return p;
}

void set_pages(CacheParams& p, const int* page_table, int page_size, int max_pages, int num_pages) {
  p.page_table = page_table;
  p.slab = page_size;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
}

}  // namespace

extern "C" int kv_write_contig(const void* k_new, const void* v_new, long long k_stride, long long v_stride,
                               const int* seq_lens, int batch, int q_len, int num_kv_heads, int head_dim, int max_ctx,
                               const double* inv_freq, int rot_offset, int rot_dim, int interleaved, float magnitude,
                               void* k, void* v, void* stream) {
  CacheParams p = write_params(k_new, v_new, k_stride, v_stride, seq_lens, batch, q_len, num_kv_heads, head_dim,
                               inv_freq, rot_offset, rot_dim, interleaved, magnitude, k, v, nullptr, nullptr);
  p.slab = max_ctx;
  return write_call(false, false, p, max_ctx, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int kv_write_paged(const void* k_new, const void* v_new, long long k_stride, long long v_stride,
                              const int* page_table, const int* seq_lens, int batch, int q_len, int num_kv_heads,
                              int head_dim, int page_size, int max_pages_per_seq, int num_pages, int max_seq_len,
                              const double* inv_freq, int rot_offset, int rot_dim, int interleaved, float magnitude,
                              void* k_pool, void* v_pool, void* stream) {
  CacheParams p = write_params(k_new, v_new, k_stride, v_stride, seq_lens, batch, q_len, num_kv_heads, head_dim,
                               inv_freq, rot_offset, rot_dim, interleaved, magnitude, k_pool, v_pool, nullptr, nullptr);
  set_pages(p, page_table, page_size, max_pages_per_seq, num_pages);
  return write_call(true, false, p, paged_cap(page_size, max_pages_per_seq, max_seq_len),
                    reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int kv_write_int8_contig(const void* k_new, const void* v_new, long long k_stride, long long v_stride,
                                    const int* seq_lens, int batch, int q_len, int num_kv_heads, int head_dim,
                                    int max_ctx, const double* inv_freq, int rot_offset, int rot_dim, int interleaved,
                                    float magnitude, void* k_i8, void* v_i8, float* k_scale, float* v_scale,
                                    void* stream) {
  CacheParams p = write_params(k_new, v_new, k_stride, v_stride, seq_lens, batch, q_len, num_kv_heads, head_dim,
                               inv_freq, rot_offset, rot_dim, interleaved, magnitude, k_i8, v_i8, k_scale, v_scale);
  p.slab = max_ctx;
  return write_call(false, true, p, max_ctx, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int kv_write_int8_paged(const void* k_new, const void* v_new, long long k_stride, long long v_stride,
                                   const int* page_table, const int* seq_lens, int batch, int q_len, int num_kv_heads,
                                   int head_dim, int page_size, int max_pages_per_seq, int num_pages, int max_seq_len,
                                   const double* inv_freq, int rot_offset, int rot_dim, int interleaved,
                                   float magnitude, void* k_pool_i8, void* v_pool_i8, float* k_scale_pool,
                                   float* v_scale_pool, void* stream) {
  CacheParams p =
      write_params(k_new, v_new, k_stride, v_stride, seq_lens, batch, q_len, num_kv_heads, head_dim, inv_freq,
                   rot_offset, rot_dim, interleaved, magnitude, k_pool_i8, v_pool_i8, k_scale_pool, v_scale_pool);
  set_pages(p, page_table, page_size, max_pages_per_seq, num_pages);
  return write_call(true, true, p, paged_cap(page_size, max_pages_per_seq, max_seq_len),
                    reinterpret_cast<cudaStream_t>(stream));
}

namespace {

int read_contig_int8(const void* k_i8, const void* v_i8, const float* k_scale, const float* v_scale, const int* starts,
                     const int* seq_lens, int batch, int n_tokens, int num_kv_heads, int head_dim, int max_ctx,
                     void* k_out, void* v_out, void* stream, bool fill) {
  CacheParams p = read_params(k_i8, v_i8, k_scale, v_scale, starts, seq_lens, batch, n_tokens, num_kv_heads, head_dim,
                              k_out, v_out, fill);
  p.slab = max_ctx;
  return read_call(false, true, p, max_ctx, reinterpret_cast<cudaStream_t>(stream));
}

int read_paged(bool int8, const void* k, const void* v, const float* ks, const float* vs, const int* page_table,
               const int* starts, const int* seq_lens, int batch, int n_tokens, int num_kv_heads, int head_dim,
               int page_size, int max_pages, int num_pages, int max_seq_len, void* k_out, void* v_out, void* stream,
               bool fill) {
  CacheParams p = read_params(k, v, ks, vs, starts, seq_lens, batch, n_tokens, num_kv_heads, head_dim, k_out, v_out,
                              fill);
  set_pages(p, page_table, page_size, max_pages, num_pages);
  return read_call(true, int8, p, paged_cap(page_size, max_pages, max_seq_len), reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" int kv_read_int8_contig(const void* k_i8, const void* v_i8, const float* k_scale, const float* v_scale,
                                   const int* starts, const int* seq_lens, int batch, int n_tokens, int num_kv_heads,
                                   int head_dim, int max_ctx, void* k_out, void* v_out, void* stream) {
  return read_contig_int8(k_i8, v_i8, k_scale, v_scale, starts, seq_lens, batch, n_tokens, num_kv_heads, head_dim,
                          max_ctx, k_out, v_out, stream, false);
}

extern "C" int kv_read_paged(const void* k_pool, const void* v_pool, const int* page_table, const int* starts,
                             const int* seq_lens, int batch, int n_tokens, int num_kv_heads, int head_dim,
                             int page_size, int max_pages_per_seq, int num_pages, int max_seq_len, void* k_out,
                             void* v_out, void* stream) {
  return read_paged(false, k_pool, v_pool, nullptr, nullptr, page_table, starts, seq_lens, batch, n_tokens,
                    num_kv_heads, head_dim, page_size, max_pages_per_seq, num_pages, max_seq_len, k_out, v_out, stream,
                    false);
}

extern "C" int kv_read_int8_paged(const void* k_pool_i8, const void* v_pool_i8, const float* k_scale_pool,
                                  const float* v_scale_pool, const int* page_table, const int* starts,
                                  const int* seq_lens, int batch, int n_tokens, int num_kv_heads, int head_dim,
                                  int page_size, int max_pages_per_seq, int num_pages, int max_seq_len, void* k_out,
                                  void* v_out, void* stream) {
  return read_paged(true, k_pool_i8, v_pool_i8, k_scale_pool, v_scale_pool, page_table, starts, seq_lens, batch,
                    n_tokens, num_kv_heads, head_dim, page_size, max_pages_per_seq, num_pages, max_seq_len, k_out,
                    v_out, stream, false);
}

extern "C" int kv_read_int8_contig_filled(const void* k_i8, const void* v_i8, const float* k_scale,
                                          const float* v_scale, const int* starts, const int* seq_lens, int batch,
                                          int n_tokens, int num_kv_heads, int head_dim, int max_ctx, void* k_out,
                                          void* v_out, void* stream) {
  return read_contig_int8(k_i8, v_i8, k_scale, v_scale, starts, seq_lens, batch, n_tokens, num_kv_heads, head_dim,
                          max_ctx, k_out, v_out, stream, true);
}

extern "C" int kv_read_paged_filled(const void* k_pool, const void* v_pool, const int* page_table, const int* starts,
                                    const int* seq_lens, int batch, int n_tokens, int num_kv_heads, int head_dim,
                                    int page_size, int max_pages_per_seq, int num_pages, int max_seq_len, void* k_out,
                                    void* v_out, void* stream) {
  return read_paged(false, k_pool, v_pool, nullptr, nullptr, page_table, starts, seq_lens, batch, n_tokens,
                    num_kv_heads, head_dim, page_size, max_pages_per_seq, num_pages, max_seq_len, k_out, v_out, stream,
                    true);
}

extern "C" int kv_read_int8_paged_filled(const void* k_pool_i8, const void* v_pool_i8, const float* k_scale_pool,
                                         const float* v_scale_pool, const int* page_table, const int* starts,
                                         const int* seq_lens, int batch, int n_tokens, int num_kv_heads, int head_dim,
                                         int page_size, int max_pages_per_seq, int num_pages, int max_seq_len,
                                         void* k_out, void* v_out, void* stream) {
  return read_paged(true, k_pool_i8, v_pool_i8, k_scale_pool, v_scale_pool, page_table, starts, seq_lens, batch,
                    n_tokens, num_kv_heads, head_dim, page_size, max_pages_per_seq, num_pages, max_seq_len, k_out,
                    v_out, stream, true);
}
