// Logit constraints ("Softmax-free GPU sampling: Gumbel-max categorical
// sampling kernel", lablup/mlxcel issue #900, Background: the token bias and
// the repetition / frequency / presence penalties ahead of the sampler; and
// grammar masks): the per-request state and the kernel that writes the
// constrained logits. The draw from them is the samplers' own (sample_kernel
// and sample_cluster_kernel with CON).
#include <climits>
#include <cstdint>

#include <cuda_bf16.h>

#include "gsample_constrain.cuh"
#include "gsample_internal.h"

namespace gsample {
namespace {

constexpr int kConThreads = 256;

// ---------------------------------------------------------------------------
// State
// ---------------------------------------------------------------------------
__device__ __forceinline__ int64_t state_row(const StateArgs& s, const int32_t* slot, int64_t i) {
  const int64_t r = slot ? (int64_t)__ldg(slot + i) : i;
  return r >= 0 && r < s.rows ? r : -1;
}

// One thread per touched word: a word without bits costs its read alone.
__global__ void __launch_bounds__(kConThreads) state_reset_kernel(const StateArgs s,
                                                                  const int32_t* slot, int64_t n) {
  pdl_wait_then_release();
  const int64_t words = s.ld / 32, total = n * words;
  for (int64_t j = blockIdx.x * (int64_t)kConThreads + threadIdx.x; j < total;
       j += (int64_t)gridDim.x * kConThreads) {
    const int64_t i = j / words, w = j - i * words;
    const int64_t r = state_row(s, slot, i);
    if (r < 0) continue;
    uint32_t* word = s.touched + r * words + w;
    const uint32_t bits = __ldcg(word);
    if (bits == 0u) continue;
    const int64_t e0 = r * s.ld + w * 32;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if ((bits >> (4 * q)) & 0xFu) {
        *reinterpret_cast<uint4*>(s.history + e0 + 4 * q) = zero;
        if (s.bias) *reinterpret_cast<uint4*>(s.bias + e0 + 4 * q) = zero;
      }
    }
    *word = 0u;
  }
}

// The request that owns list position j: the last i with offsets[i] <= j, or
// -1 when j lies outside every request.
__device__ __forceinline__ int64_t owner(const int64_t* offsets, int64_t n, int64_t j) {
  if (!offsets) return j;
  if (j < __ldg(offsets) || j >= __ldg(offsets + n)) return -1;
  int64_t lo = 0, hi = n;  // offsets[lo] <= j < offsets[hi]
  while (hi - lo > 1) {
    const int64_t mid = lo + (hi - lo) / 2;
    if (__ldg(offsets + mid) <= j)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// One thread per token. Integer atomics commute, so the state does not depend
// on their order.
__global__ void __launch_bounds__(kConThreads)
    history_append_kernel(const StateArgs s, const int32_t* slot, int64_t n, const int64_t* tokens,
                          int64_t total, const int64_t* offsets, bool prompt) {
  pdl_wait_then_release();
  for (int64_t j = blockIdx.x * (int64_t)kConThreads + threadIdx.x; j < total;
       j += (int64_t)gridDim.x * kConThreads) {
    const int64_t t = __ldg(tokens + j);
    const int64_t i = owner(offsets, n, j);
    if (i < 0 || t < 0 || t >= s.vocab) continue;
    const int64_t r = state_row(s, slot, i);
    if (r < 0) continue;
    uint32_t* h = s.history + r * s.ld + t;
    const uint32_t before = prompt ? atomicOr(h, 0x80000000u) : atomicAdd(h, 1u);
    if (before == 0u) atomicOr(s.touched + r * (s.ld / 32) + (t >> 5), 1u << (t & 31));
  }
}

// One warp per request walks its list 32 entries at a time; of the entries of
// a step that name the same token the last one writes, and later steps
// overwrite earlier ones, so the later value stays.
__global__ void __launch_bounds__(32)
    bias_set_kernel(const StateArgs s, const int32_t* slot, const int64_t* tokens,
                    const float* values, int64_t total, const int64_t* offsets) {
  pdl_wait_then_release();
  const int64_t i = blockIdx.x;
  const int lane = threadIdx.x;
  const int64_t r = state_row(s, slot, i);
  if (r < 0) return;
  int64_t lo = offsets ? __ldg(offsets + i) : i;
  int64_t hi = offsets ? __ldg(offsets + i + 1) : i + 1;
  lo = lo < 0 ? 0 : lo;
  hi = hi > total ? total : hi;
  for (int64_t j0 = lo; j0 < hi; j0 += 32) {
    const int64_t j = j0 + lane;
    int64_t t = -1;
    float v = 0.0f;
    if (j < hi) {
      t = __ldg(tokens + j);
      v = __ldg(values + j);
      if (t < 0 || t >= s.vocab) t = -1;
    }
    const unsigned same = __match_any_sync(0xFFFFFFFFu, (unsigned long long)t);
    if (t >= 0 && lane == 31 - __clz(same)) {
      s.bias[r * s.ld + t] = v;
      atomicOr(s.touched + r * (s.ld / 32) + (t >> 5), 1u << (t & 31));
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// Constrained logits
// ---------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ float load_one(const char* row, int32_t i) {
  if constexpr (DT == 0) return reinterpret_cast<const float*>(row)[i];
  const uint32_t h = reinterpret_cast<const unsigned short*>(row)[i];
  return half_to_f32<DT>(h);
}

template <int DT>
__device__ __forceinline__ void store_one(char* row, int32_t i, float x) {
  if constexpr (DT == 0) {
    reinterpret_cast<float*>(row)[i] = x;
  } else if constexpr (DT == 1) {
    reinterpret_cast<__nv_bfloat16*>(row)[i] = __float2bfloat16_rn(x);
  } else {
    reinterpret_cast<__half*>(row)[i] = __float2half_rn(x);
  }
}

template <int DT, int ODT>
__global__ void __launch_bounds__(kConThreads) process_kernel(const ProcessParams p) {
  pdl_wait_then_release();
  const int64_t cpr = (p.V + kConThreads - 1) / kConThreads;
  const bool inplace = p.inplace;
  for (int64_t c = blockIdx.x; c < p.B * cpr; c += gridDim.x) {
    const int64_t b = c / cpr;
    const int64_t v = (c - b * cpr) * kConThreads + threadIdx.x;
    if (v >= p.V) continue;
    const RowConstraints r = row_constraints(p.con, b);
    const float x = load_one<DT>(p.logits + b * p.ld_bytes, (int32_t)v);
    const float y = constrained_logit(x, (int32_t)v, r);
    if (!inplace || __float_as_uint(x) != __float_as_uint(y))
      store_one<ODT>(p.out + b * p.out_ld_bytes, (int32_t)v, y);
  }
}

// Launch with programmatic stream serialization, as every kernel here.
template <typename... Params, typename... Args>
cudaError_t launch(void (*fn)(Params...), int64_t blocks, int threads, cudaStream_t stream,
                   Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<Params>(args)...);
}

int64_t blocks_for(int64_t items, int64_t per_block, int64_t most) {
  const int64_t n = (items + per_block - 1) / per_block;
  return n < 1 ? 1 : n > most ? most : n;
}

}  // namespace

cudaError_t launch_state_reset(const StateArgs& s, const int32_t* slot, int64_t n, int sms,
                               cudaStream_t stream) {
  const int64_t blocks = blocks_for(n * (s.ld / 32), kConThreads, (int64_t)sms * 8);
  return launch(state_reset_kernel, blocks, kConThreads, stream, s, slot, n);
}

cudaError_t launch_history_append(const StateArgs& s, const int32_t* slot, int64_t n,
                                  const int64_t* tokens, int64_t total, const int64_t* offsets,
                                  bool prompt, int sms, cudaStream_t stream) {
  const int64_t blocks = blocks_for(total, kConThreads, (int64_t)sms * 8);
  return launch(history_append_kernel, blocks, kConThreads, stream, s, slot, n, tokens, total,
                offsets, prompt);
}

cudaError_t launch_bias_set(const StateArgs& s, const int32_t* slot, int64_t n,
                            const int64_t* tokens, const float* values, int64_t total,
                            const int64_t* offsets, cudaStream_t stream) {
  return launch(bias_set_kernel, n, 32, stream, s, slot, tokens, values, total, offsets);
}

cudaError_t launch_process(const ProcessParams& p, int dtype, int out_dtype, int sms,
                           cudaStream_t stream) {
  const int64_t cpr = (p.V + kConThreads - 1) / kConThreads;
  const int64_t blocks = blocks_for(p.B * cpr, 1, (int64_t)sms * 8);
  switch (dtype * 2 + (out_dtype == 0 ? 0 : 1)) {
    case 0: return launch(process_kernel<0, 0>, blocks, kConThreads, stream, p);
    case 2: return launch(process_kernel<1, 0>, blocks, kConThreads, stream, p);
    case 3: return launch(process_kernel<1, 1>, blocks, kConThreads, stream, p);
    case 4: return launch(process_kernel<2, 0>, blocks, kConThreads, stream, p);
    default: return launch(process_kernel<2, 2>, blocks, kConThreads, stream, p);
  }
}

}  // namespace gsample
