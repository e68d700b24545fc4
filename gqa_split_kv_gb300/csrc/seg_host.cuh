// Host side of seg_kernel.cuh: grid, partials and launch.
#pragma once

#include <atomic>

#include "host_util.cuh"
#include "seg_kernel.cuh"

namespace da {
namespace {

// Query rows of a unit, of `rows` a KV head: 8 where that is all or, at D = 256, where 16 would leave an SM one CTA's
// registers; else 16, which read a key and value once.
int seg_unit_rows(long long rows, int D) { return rows <= 8 || D == 256 ? 8 : 16; }

// CTAs of seg_kernel: as many as run at once.
int seg_ctas(int ru, int D, int sms) {
  const int per_sm = ru == 8 ? (D == 64 ? SegGeo<64, 1>::PER_SM : D == 128 ? SegGeo<128, 1>::PER_SM : SegGeo<256, 1>::PER_SM)
                             : (D == 64 ? SegGeo<64, 2>::PER_SM : SegGeo<128, 2>::PER_SM);
  return sms * per_sm;
}

long long seg_partial_bytes(long long slots, int ru, int D) { return slots * ru * (D * 4ll + 8); }

void seg_partials(SegParams& p, void* workspace, long long slots, int D) {
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + slots * p.ru * D);
}

// Tokens that a paged cache of a sequence can hold (what the sizes allow, max_seq_len at most).
long long capacity(int page_size, int max_pages, int max_seq_len) {
  if (page_size <= 0 || max_pages < 0) return 0;
  const long long room = (long long)max_pages * page_size;
  return room < max_seq_len ? room : max_seq_len;
}

// Lets a kernel use this much shared memory, once a device.
template <auto KERN, bool CLUSTERS_OF_16 = false>
int allow_smem(size_t bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev;
  if (current_device(&dev) || dev >= kMaxDevices) return DA_ERR_CUDA;
  if (done.load(std::memory_order_relaxed) >> dev & 1) return DA_OK;
  if (cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess ||
      cudaFuncSetAttribute(KERN, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
          cudaSuccess ||
      (CLUSTERS_OF_16 && cudaFuncSetAttribute(KERN, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)) {
    cudaGetLastError();
    return DA_ERR_CUDA;
  }
  done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return DA_OK;
}

// launch_dependent in clusters of this many CTAs.
template <typename P>
int launch_clusters(void (*kern)(P), unsigned grid, unsigned threads, size_t smem, int cluster, cudaStream_t st,
                    const P& prm) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, prm) != cudaSuccess) {
    cudaGetLastError();
    return DA_ERR_CUDA;
  }
  return DA_OK;
}

template <int D, bool PAGED, int KIND, int NT>
int launch_seg_nt(const SegParams& p, cudaStream_t st) {
  using Gm = SegGeo<D, NT, KIND>;
  if (int e = allow_smem<seg_kernel<D, PAGED, KIND, NT>, KIND == kSegBlocks>(Gm::SMEM)) return e;
  if (KIND == kSegBlocks)
    return launch_clusters(seg_kernel<D, PAGED, KIND, NT>, (unsigned)p.ctas, Gm::THREADS, Gm::SMEM, p.cluster, st, p);
  return launch_dependent(seg_kernel<D, PAGED, KIND, NT>, (unsigned)p.ctas, Gm::THREADS, Gm::SMEM, st, p);
}
template <int D, bool PAGED, int KIND>
int launch_seg(const SegParams& p, cudaStream_t st) {
  if constexpr (D != 256)
    if (p.ru == 16) return launch_seg_nt<D, PAGED, KIND, 2>(p, st);
  return launch_seg_nt<D, PAGED, KIND, 1>(p, st);
}

}  // namespace
}  // namespace da
