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

// The row kernel. Row b of the result is cut into units of N elements (N = 8
// for 16-bit logits, 4 for binary32: 16 bytes of the logits) that start on
// 16-byte boundaries of the RESULT, so that every full unit is stored with
// 128-bit stores wherever the two rows start; the first and last unit may be
// partial and go element by element. The logits of a full unit are one 128-bit
// load where they are aligned too; otherwise the two aligned 16-byte pieces
// that hold them, shifted together (both inside the row: units for which they
// are not count as partial). ALIGNED: both matrices' rows all start on 16-byte
// boundaries.
//
// A warp works alone, on kBatch runs of 32 units at a time that lie
// warps_per_row runs apart: the low ids, which hold most of a request's
// tokens, are shared by many warps. First the mask and touched bits, then the
// units that the mask leaves anything of (the others are never read), then
// their stores; then the touched elements, listed in shared memory, are
// fetched again with their state words and written over their places, one a
// lane.
//
// In place, a unit is read and written only where the mask takes some but not
// all of it, written only where it takes all, and touched elements are the only
// traffic elsewhere.
#ifndef GSAMPLE_PROCESS_CTAS
#define GSAMPLE_PROCESS_CTAS 4
#endif
#ifndef GSAMPLE_PROCESS_RUNS
#define GSAMPLE_PROCESS_RUNS 8
#endif
constexpr int kBatch = 4;
constexpr int kTouchedCap = 256;  // elements a warp lists at a time

__device__ __forceinline__ uint4 ld_unit(const char* p, uint64_t pol) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(pol)
               : "memory");
  return v;
}

// 16 bytes at p, `a` (0 < a < 16) bytes past a 16-byte boundary.
__device__ __forceinline__ uint4 ld_unit_shifted(const char* p, int a, uint64_t pol) {
  const uint4 lo = ld_unit(p - a, pol), hi = ld_unit(p - a + 16, pol);
  const int sh = (a & 3) * 8;
  uint32_t w[5];
  switch (a >> 2) {  // the same for a whole row
    case 0: w[0] = lo.x; w[1] = lo.y; w[2] = lo.z; w[3] = lo.w; w[4] = hi.x; break;
    case 1: w[0] = lo.y; w[1] = lo.z; w[2] = lo.w; w[3] = hi.x; w[4] = hi.y; break;
    case 2: w[0] = lo.z; w[1] = lo.w; w[2] = hi.x; w[3] = hi.y; w[4] = hi.z; break;
    default: w[0] = lo.w; w[1] = hi.x; w[2] = hi.y; w[3] = hi.z; w[4] = hi.w; break;
  }
  return make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh),
                    __funnelshift_r(w[2], w[3], sh), __funnelshift_r(w[3], w[4], sh));
}

// The N bits of a bit row from bit e0 on; all of them lie inside the row.
template <int N>
__device__ __forceinline__ uint32_t bits_at(const uint8_t* bits, int32_t e0) {
  const int sh = e0 & 7;
  uint32_t v = __ldcg(bits + (e0 >> 3));
  if (sh + N > 8) v |= (uint32_t)__ldcg(bits + (e0 >> 3) + 1) << 8;
  return (v >> sh) & ((1u << N) - 1u);
}

template <int DT, int ODT, bool INPLACE, bool ALIGNED>
__global__ void __launch_bounds__(kConThreads, GSAMPLE_PROCESS_CTAS)
    process_kernel(const ProcessParams p) {
  constexpr int N = DT == 0 ? 4 : 8;
  constexpr int ISZ = DT == 0 ? 4 : 2, OSZ = ODT == 0 ? 4 : 2;
  constexpr uint32_t kFull = (1u << N) - 1u;
  __shared__ uint32_t lists[kConThreads / 32][kTouchedCap];
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t Q = p.warps_per_row;
  const int32_t q = (int32_t)blockIdx.x * (kConThreads / 32) + warp;
  if (q >= Q) return;
  uint32_t* list = lists[warp];
  const uint64_t pol = evict_first_policy();
  const int32_t V = (int32_t)p.V;
  for (int64_t b = blockIdx.y; b < p.B; b += gridDim.y) {
    const RowBits r = row_bits(p.con, b);
    const char* in = p.logits + b * p.ld_bytes;
    char* out = p.out + b * p.out_ld_bytes;
    // Elements by which unit 0 starts before the row, and the misalignment of
    // the logits of every unit.
    const int32_t s = ALIGNED ? 0 : (int32_t)((uintptr_t)out & 15u) / OSZ;
    const int a = ALIGNED ? 0 : (int)(((uintptr_t)in - (uintptr_t)(s * ISZ)) & 15u);
    // Full units start in [lo, hi]: all N elements lie in the row, and every
    // byte that is loaded for them (a multiple of ISZ before and after).
    const int32_t lo = a / ISZ, hi = V - (a == 0 ? N : (32 - a) / ISZ);
#pragma unroll 1
    for (int32_t run = q; run < p.runs_per_row; run += kBatch * Q) {
      int32_t e0[kBatch];
      uint32_t allowed[kBatch], touched[kBatch];
      bool full[kBatch], partial = false;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int32_t u = (run + k * Q) * 32 + lane;
        const bool in_row = run + k * Q < p.runs_per_row && u < p.units_per_row;
        e0[k] = in_row ? u * N - s : V;  // V: neither full nor partial
        full[k] = in_row && e0[k] >= lo && e0[k] <= hi;
        partial |= in_row && !full[k];
        allowed[k] = 0u;
        touched[k] = 0u;
        if (full[k]) {
          if constexpr (ALIGNED) {
            allowed[k] = r.mask ? unit_bits<N>(r.mask, e0[k]) : kFull;
            if (r.touched) touched[k] = unit_bits<N>(r.touched, e0[k]);
          } else {
            allowed[k] = r.mask ? bits_at<N>(r.mask, e0[k]) : kFull;
            if (r.touched) touched[k] = bits_at<N>(r.touched, e0[k]);
          }
        }
      }
      uint4 x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const char* at = in + (int64_t)e0[k] * ISZ;
        if (allowed[k] != 0u && (!INPLACE || allowed[k] != kFull))
          x[k] = a == 0 ? ld_unit(at, pol) : ld_unit_shifted(at, a, pol);
      }
      uint32_t todo = 0u;  // the lane's touched elements, N bits a unit
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (!full[k]) continue;
        todo |= (touched[k] & allowed[k]) << (N * k);
        if (INPLACE && allowed[k] == kFull) continue;
        const uint4 y = allowed[k] == kFull ? x[k] : masked_unit<DT, DT == 0>(x[k], allowed[k]);
        uint4* dst = reinterpret_cast<uint4*>(out + (int64_t)e0[k] * OSZ);
        if constexpr (DT != 0 && ODT == 0) {
          const uint32_t w[4] = {y.x, y.y, y.z, y.w};
          float f[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[2 * i] = half_to_f32<DT>(w[i] & 0xFFFFu);
            f[2 * i + 1] = half_to_f32<DT>(w[i] >> 16);
          }
          dst[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                              __float_as_uint(f[3]));
          dst[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                              __float_as_uint(f[7]));
        } else {
          dst[0] = y;
        }
      }
      static_assert(N * kBatch <= 32, "a lane's touched bits fit in one word");
      if (__any_sync(0xFFFFFFFFu, todo != 0u)) {
        int incl = __popc(todo);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
          if (lane >= o) incl += up;
        }
        const int total = __shfl_sync(0xFFFFFFFFu, incl, 31);
        const int first = incl - __popc(todo);
#pragma unroll 1
        for (int base = 0; base < total; base += kTouchedCap) {
          int at = first - base;
          for (uint32_t bits = todo; bits != 0u; bits &= bits - 1u, ++at) {
            const int j = __ffs((int)bits) - 1;
            if (at >= 0 && at < kTouchedCap)
              list[at] = (uint32_t)(((run + j / N * Q) * 32 + lane) * N - s + j % N);
          }
          __syncwarp();  // also orders the units' stores before these elements'
          const int n = min(kTouchedCap, total - base);
          // The next element's gathers are on their way while one is written.
          int32_t v_next = 0;
          float l_next = 0.0f, bias_next = 0.0f;
          uint32_t h_next = 0u;
          auto gather = [&](int i) {
            if (i >= n) return;
            v_next = (int32_t)list[i];
            l_next = load_one<DT>(in, v_next);
            h_next = __ldcg(p.con.history + r.state + v_next);
            if (p.con.bias) bias_next = __ldcg(p.con.bias + r.state + v_next);
          };
          gather(lane);
          const RowPenalties pen = row_penalties(p.con, b);
#pragma unroll 1
          for (int i = lane; i < n; i += 32) {
            const int32_t v = v_next;
            const float l = l_next, bias = bias_next;
            const uint32_t h = h_next;
            gather(i + 32);
            store_one<ODT>(out, v, penalised(l, h, bias, pen));
          }
          __syncwarp();
        }
      }
      if (partial) {  // the units at the row's ends
#pragma unroll 1
        for (int k = 0; k < kBatch; ++k) {
          const int32_t u = (run + k * Q) * 32 + lane;
          if (run + k * Q >= p.runs_per_row || u >= p.units_per_row) break;
          const int32_t e = u * N - s;
          if (e >= lo && e <= hi) continue;
          for (int32_t v = e < 0 ? 0 : e; v < e + N && v < V; ++v) {
            const float l = load_one<DT>(in, v);
            const float y = constrained_logit(l, v, row_constraints(p.con, b));
            if (!INPLACE || __float_as_uint(l) != __float_as_uint(y)) store_one<ODT>(out, v, y);
          }
        }
      }
      __syncwarp();
    }
  }
}

// Launch with programmatic stream serialization, as every kernel here.
template <typename... Params, typename... Args>
cudaError_t launch(void (*fn)(Params...), dim3 grid, int threads, cudaStream_t stream,
                   Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<Params>(args)...);
}

dim3 blocks_for(int64_t items, int64_t per_block, int64_t most) {
  const int64_t n = (items + per_block - 1) / per_block;
  return dim3((unsigned)(n < 1 ? 1 : n > most ? most : n));
}

}  // namespace

cudaError_t launch_state_reset(const StateArgs& s, const int32_t* slot, int64_t n, int sms,
                               cudaStream_t stream) {
  const dim3 blocks = blocks_for(n * (s.ld / 32), kConThreads, (int64_t)sms * 8);
  return launch(state_reset_kernel, blocks, kConThreads, stream, s, slot, n);
}

cudaError_t launch_history_append(const StateArgs& s, const int32_t* slot, int64_t n,
                                  const int64_t* tokens, int64_t total, const int64_t* offsets,
                                  bool prompt, int sms, cudaStream_t stream) {
  const dim3 blocks = blocks_for(total, kConThreads, (int64_t)sms * 8);
  return launch(history_append_kernel, blocks, kConThreads, stream, s, slot, n, tokens, total,
                offsets, prompt);
}

cudaError_t launch_bias_set(const StateArgs& s, const int32_t* slot, int64_t n,
                            const int64_t* tokens, const float* values, int64_t total,
                            const int64_t* offsets, cudaStream_t stream) {
  return launch(bias_set_kernel, dim3((unsigned)n), 32, stream, s, slot, tokens, values, total, offsets);
}

cudaError_t launch_process(ProcessParams p, int dtype, int out_dtype, int sms,
                           cudaStream_t stream) {
  // One unit more than the elements need where the first may start before the
  // row. A warp takes up to GSAMPLE_PROCESS_RUNS runs of a row, fewer while
  // there are not enough warps to fill the device.
  const int64_t n = dtype == 0 ? 4 : 8;
  const bool aligned = (((uintptr_t)p.logits | (uintptr_t)p.out | (uintptr_t)p.ld_bytes |
                         (uintptr_t)p.out_ld_bytes) & 15u) == 0;
  const int64_t units = (p.V + n - 1) / n + (aligned ? 0 : 1);
  const int64_t runs = (units + 31) / 32;
  int64_t per_warp = GSAMPLE_PROCESS_RUNS;
  const int64_t slots = (int64_t)sms * GSAMPLE_PROCESS_CTAS * (kConThreads / 32);
  while (per_warp > 1 && p.B * ((runs + per_warp - 1) / per_warp) < slots) per_warp /= 2;
  p.units_per_row = (int32_t)units;
  p.runs_per_row = (int32_t)runs;
  p.warps_per_row = (int32_t)((runs + per_warp - 1) / per_warp);
  const int64_t bx = (p.warps_per_row + kConThreads / 32 - 1) / (kConThreads / 32);
  const dim3 grid((unsigned)bx, (unsigned)(p.B < 65535 ? p.B : 65535));
  switch (dtype * 8 + (out_dtype == 0 ? 0 : 4) + (p.inplace ? 2 : 0) + (aligned ? 1 : 0)) {
    case 0: return launch(process_kernel<0, 0, false, false>, grid, kConThreads, stream, p);
    case 1: return launch(process_kernel<0, 0, false, true>, grid, kConThreads, stream, p);
    case 2: return launch(process_kernel<0, 0, true, false>, grid, kConThreads, stream, p);
    case 3: return launch(process_kernel<0, 0, true, true>, grid, kConThreads, stream, p);
    case 8: return launch(process_kernel<1, 0, false, false>, grid, kConThreads, stream, p);
    case 9: return launch(process_kernel<1, 0, false, true>, grid, kConThreads, stream, p);
    case 12: return launch(process_kernel<1, 1, false, false>, grid, kConThreads, stream, p);
    case 13: return launch(process_kernel<1, 1, false, true>, grid, kConThreads, stream, p);
    case 14: return launch(process_kernel<1, 1, true, false>, grid, kConThreads, stream, p);
    case 15: return launch(process_kernel<1, 1, true, true>, grid, kConThreads, stream, p);
    case 16: return launch(process_kernel<2, 0, false, false>, grid, kConThreads, stream, p);
    case 17: return launch(process_kernel<2, 0, false, true>, grid, kConThreads, stream, p);
    case 20: return launch(process_kernel<2, 2, false, false>, grid, kConThreads, stream, p);
    case 21: return launch(process_kernel<2, 2, false, true>, grid, kConThreads, stream, p);
    case 22: return launch(process_kernel<2, 2, true, false>, grid, kConThreads, stream, p);
    default: return launch(process_kernel<2, 2, true, true>, grid, kConThreads, stream, p);
  }
}

}  // namespace gsample
