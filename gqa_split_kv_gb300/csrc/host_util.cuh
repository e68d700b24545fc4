// Host helpers that every translation unit of the library uses: the current
// device's limits, the TMA map encoder and pointer alignment.  Each unit holds its
// own copy (internal linkage), so the units need nothing of each other.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/decode_attn.h"

namespace da {
namespace {

constexpr int kMaxDevices = 64;
constexpr unsigned long long kWaitTimeoutNs = 2000000000ull;  // 2 s per bounded wait

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

std::mutex g_mu;
EncodeTiledFn g_encode = nullptr;
int g_num_sms[kMaxDevices] = {0};
int g_smem_optin[kMaxDevices] = {0};

int current_device(int* dev) { return cudaGetDevice(dev) == cudaSuccess ? DA_OK : DA_ERR_CUDA; }

int device_info(int dev, int* sms, int* smem_optin) {
  if (dev < 0 || dev >= kMaxDevices) return DA_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_num_sms[dev] == 0) {
    int s = 0, m = 0;
    if (cudaDeviceGetAttribute(&s, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&m, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess) {
      cudaGetLastError();
      return DA_ERR_CUDA;
    }
    g_num_sms[dev] = s;
    g_smem_optin[dev] = m;
  }
  *sms = g_num_sms[dev];
  *smem_optin = g_smem_optin[dev];
  return DA_OK;
}

int get_encoder(EncodeTiledFn* fn) {
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_encode) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess || p == nullptr) {
      cudaGetLastError();
      return DA_ERR_CUDA;
    }
    g_encode = reinterpret_cast<EncodeTiledFn>(p);
  }
  *fn = g_encode;
  return DA_OK;
}

// Tiled map; dims/box innermost first, strides in bytes for dims 1..rank-1.
int encode_map_t(CUtensorMap* m, CUtensorMapDataType type, CUtensorMapSwizzle swz, const void* base, int rank,
                 const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  EncodeTiledFn enc;
  if (int st = get_encoder(&enc)) return st;
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = enc(m, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DA_OK : DA_ERR_INVALID_ARG;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether a tensor can have n steps of this stride (in elements): 2^56 of them at most, more than any memory
// holds, so that sums and byte counts of such extents stay in 64 bits.
bool reachable(long long n, long long stride) {
  return stride >= 0 && (stride == 0 || n <= (1LL << 56) / stride);
}

// The product of sizes that are not negative, at most 2^60.
template <typename... T>
long long product(T... n) {
  long long p = 1;
  for (long long x : {(long long)n...}) p = x == 0 || p == 0 ? 0 : p > (1LL << 60) / x ? 1LL << 60 : p * x;
  return p;
}

// Whether [a, a + an) and [b, b + bn) share a byte (null pointers: no).
bool overlap(const void* a, long long an, const void* b, long long bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && an > 0 && bn > 0 && x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

// Launches kern as a programmatic dependent of what precedes it in the stream: its CTAs may
// start while that drains, so every kernel launched here waits for it (griddepcontrol.wait)
// before it touches memory that an earlier kernel may write or read, and reads such memory
// by load_dependent or __ldcg, never through the read-only path.  Some touch memory earlier, where their only
// predecessor lets them start after its own wait (so all kernels before that one are done) and does not write
// what they read, nor use what they write:
//   latent_combine_kernel, seg_merge_prefix_kernel  read seq_lens,
//   weights_finish_kernel  reads lengths, page table and priors,
//   seg_kernel beside prefix_tc_kernel  reads all of its inputs and writes its own partials; it waits at its end, as
//     the kernel behind it waits for it alone.
template <typename P>
int launch_dependent(void (*kern)(P), unsigned grid, unsigned threads, size_t smem, cudaStream_t st, const P& prm) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, prm) != cudaSuccess) {
    cudaGetLastError();
    return DA_ERR_CUDA;
  }
  return DA_OK;
}

}  // namespace
}  // namespace da
