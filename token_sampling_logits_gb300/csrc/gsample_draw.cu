// Launches of the draw from given random numbers and of the verification of
// drafts; their kernels are in gsample_draw.cuh.
#include <cstdint>

#include "gsample_internal.h"
#include "gsample_weights.cuh"

namespace gsample {

void* draw_kernel_f32(bool vec, bool verify);
void* draw_kernel_bf16(bool vec, bool verify);
void* draw_kernel_f16(bool vec, bool verify);
void* verify_draw_kernel_f32(bool vec);
void* verify_draw_kernel_bf16(bool vec);
void* verify_draw_kernel_f16(bool vec);

namespace {

using u64 = unsigned long long;
constexpr int kDrawThreads = 512;  // as in gsample_draw.cuh
constexpr int kDrawMaxCluster = 16;
constexpr size_t kDrawSmemLimit = 160 * 1024;  // of the units' maxima

__global__ void __launch_bounds__(256) debug_weights_kernel(const float* x, int64_t n, float M,
                                                            float T, u64* out) {
  __shared__ float2 tab[kExp2Entries];
  for (int j = threadIdx.x; j < kExp2Entries; j += 256) tab[j] = exp2_entry(j);
  __syncthreads();
  const WeightRow w = weight_row(M, T, 0);
  for (int64_t j = blockIdx.x * (int64_t)256 + threadIdx.x; j < n; j += (int64_t)gridDim.x * 256)
    out[j] = weight_of(x[j], w, smem_addr(tab));
}

void* select_set(int dtype, bool vec, bool verify) {
  return dtype == 0   ? draw_kernel_f32(vec, verify)
         : dtype == 1 ? draw_kernel_bf16(vec, verify)
                      : draw_kernel_f16(vec, verify);
}

void* select_verify_draw(int dtype, bool vec) {
  return dtype == 0 ? verify_draw_kernel_f32(vec)
         : dtype == 1 ? verify_draw_kernel_bf16(vec) : verify_draw_kernel_f16(vec);
}

cudaError_t launch_rows(void* fn, const DrawParams& p, int64_t clusters, size_t smem,
                        cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * p.cluster));
  cfg.blockDim = dim3(kDrawThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = pdl_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  void* args[] = {const_cast<DrawParams*>(&p)};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

void* draw_kernel(int dtype, bool vec, bool verify) { return select_set(dtype, vec, verify); }
void* verify_draw_kernel_fn(int dtype, bool vec) { return select_verify_draw(dtype, vec); }
int draw_threads() { return kDrawThreads; }
size_t draw_smem_limit() { return kDrawSmemLimit; }

// One-time per-device setup of the kernels of (dtype, vec): clusters of up to
// 16 CTAs and the shared memory for the units' maxima, then the largest cluster
// that the device co-schedules.
int draw_max_cluster(int dtype, bool vec) {
  int size = kDrawMaxCluster;
  for (int v = 0; v < 3; ++v) {
    void* fn = v == 2 ? select_verify_draw(dtype, vec) : select_set(dtype, vec, v != 0);
    const int smem = v < 2 ? (int)kDrawSmemLimit : 0;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kDrawMaxCluster);
    cfg.blockDim = dim3(kDrawThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kDrawMaxCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int c = 0;
    if (cudaOccupancyMaxPotentialClusterSize(&c, fn, &cfg) != cudaSuccess) return 0;
    size = c < size ? c : size;
  }
  return size;
}

cudaError_t launch_draw(const DrawParams& p, int dtype, bool vec, int64_t clusters,
                        cudaStream_t stream) {
  return launch_rows(select_set(dtype, vec, p.sets != nullptr), p, clusters,
                     p.maxima ? draw_smem(p.units_per_cta) : 0, stream);
}

cudaError_t launch_verify_draw(const DrawParams& p, int dtype, bool vec, cudaStream_t stream) {
  return launch_rows(select_verify_draw(dtype, vec), p, p.n, 0, stream);
}

cudaError_t launch_debug_weights(const float* x, int64_t n, float M, float T, uint64_t* out,
                                 cudaStream_t stream) {
  const int64_t blocks = (n + 255) / 256;
  debug_weights_kernel<<<(unsigned)(blocks < 1024 ? blocks : 1024), 256, 0, stream>>>(
      x, n, M, T, reinterpret_cast<u64*>(out));
  return cudaGetLastError();
}

}  // namespace gsample
