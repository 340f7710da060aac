// Work split over the blocks of a cluster, for launches that leave SMs idle: the
// blocks take a share of the keys each and join their parts through the cluster's
// shared memory, so that no workspace and no second launch is needed.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "attn_kernels.h"
#include "tc_pair.cuh"

namespace rglru {

// Two or four floats of the shared memory of a block of the cluster.
__device__ __forceinline__ void ld_cluster(uint32_t addr, float &a, float &b) {
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(a), "=f"(b) : "r"(addr) : "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// The factors f_i of the parts of a row, from their maxima and sums (m, l at `ml` in
// each block; f_i O_i summed is the row), in the order of the parts:
//   M = max m_i,  L = sum l_i e^(m_i - M),  f_i = e^(m_i - M) / L
// with base 2 or e as the maxima are. A part without a key (l = 0) has factor 0: what
// lies in its O is not to be read. `sum` is L, 0 for a row that sees no key.
template <bool kBase2>
__device__ __forceinline__ void join_factors(uint32_t ml, int parts, float (&f)[8], float &top, float &sum) {
  float l[8];
  top = -INFINITY;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[i] = -INFINITY;
    l[i] = 0.0f;
    if (i < parts) ld_cluster(tc::mapa_shared(ml, i), f[i], l[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (l[i] != 0.0f) top = fmaxf(top, f[i]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[i] = l[i] == 0.0f ? 0.0f : kBase2 ? exp2f(f[i] - top) : expf(f[i] - top);
    sum += l[i] * f[i];
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = l[i] == 0.0f ? 0.0f : f[i] * inv;
}

inline cudaLaunchConfig_t cluster_config(cudaLaunchAttribute *attr, unsigned parts, dim3 grid, int threads,
                                         int smem, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = parts;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// How many clusters of 2, 4 and 8 blocks of a kernel each device runs at once, plus
// one; 0: not asked yet.
struct ClusterRoom {
  static constexpr int kMaxDev = 64;
  std::atomic<int> of[kMaxDev][3] = {};
};

// Blocks that share a unit of work: 1, or, while the units of a launch leave half of
// the SMs idle, 2, 4 or 8, `most` at most, as long as all clusters fit at once.
template <typename K>
cudaError_t cluster_parts(K kernel, int threads, int smem, std::atomic<unsigned long long> *done, ClusterRoom *room,
                          unsigned units, int most, int *parts) {
  *parts = 1;
  for (int x = 0; x < 3; ++x) {
    const int n = 2 << x;
    if (units > 148u / n || most < n) break;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int fit = dev < ClusterRoom::kMaxDev ? room->of[dev][x].load(std::memory_order_acquire) - 1 : -1;
    if (fit < 0) {
      e = opt_in_smem(kernel, smem, *done);
      if (e != cudaSuccess) return e;
      cudaLaunchAttribute attr;
      const cudaLaunchConfig_t cfg = cluster_config(&attr, n, dim3(n), threads, smem, nullptr);
      e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg);
      if (e != cudaSuccess) return e;
      if (dev < ClusterRoom::kMaxDev) room->of[dev][x].store(fit + 1, std::memory_order_release);
    }
    if (units > static_cast<unsigned>(fit)) break;
    *parts = n;
  }
  return cudaSuccess;
}

}  // namespace rglru
