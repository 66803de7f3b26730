// The constrained logit of one element, and where a batch row finds its mask,
// its state row and its parameters. Shared by the kernel that writes the
// constrained logits and the samplers that draw from them.
//
//   x == -inf stays; x += bias; x > 0 ? x / rep : x * rep for a token seen;
//   (x - freq * count) - pres for a token in the output; masked: -inf.
//
// Every operation is rounded once to binary32 (no contraction into an fma), so
// the written logits and the samplers' in-register ones are the same bits.
//
// State and mask words, and single logits, are read through L2 only (ld.cg): the
// kernel just before on the stream, which this one's start may overlap, often
// writes state words. (Whole rows of logits are read by non-coherent loads; no
// kernel that writes logits lets its successor start early.) The exact pass of
// the small-batch kernel reads the words of the elements it scores again.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>

#include "gsample_device.cuh"

namespace gsample {

// Launch-wide constraints; pointers are device memory. Bit arrays are read as
// bytes: bit v of a row is bit v & 7 of byte v >> 3 (little-endian words).
struct ConstrainArgs {
  const uint32_t* history;  // nullptr: no state
  const float* bias;        // nullptr: no biases
  const uint8_t* touched;
  int64_t state_rows;
  int64_t state_ld;  // elements, a multiple of 32
  const int32_t* slot;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const uint8_t* mask;  // nullptr: no masks
  int64_t mask_rows;
  int64_t mask_ld_bytes;
  const int32_t* mask_row;
};


// The penalties of batch row b.
struct RowPenalties {
  float rep, freq, pres;
};

__device__ __forceinline__ RowPenalties row_penalties(const ConstrainArgs& c, int64_t b) {
  RowPenalties r{1.0f, 0.0f, 0.0f};
  if (c.repetition) {
    const float v = __ldg(c.repetition + b);
    if (v > 0.0f && v < INFINITY) r.rep = v;  // NaN, <= 0 and inf: no penalty
  }
  if (c.frequency) {
    const float v = __ldg(c.frequency + b);
    if (v == v) r.freq = v;
  }
  if (c.presence) {
    const float v = __ldg(c.presence + b);
    if (v == v) r.pres = v;
  }
  return r;
}

// One batch row's view of the constraints; a null pointer means "none for this
// row".
struct RowConstraints {
  const uint8_t* mask;
  const uint8_t* touched;
  const uint32_t* history;
  const float* bias;
  RowPenalties pen;
};

// The state row of batch row b, or -1.
__device__ __forceinline__ int64_t state_row_of(const ConstrainArgs& c, int64_t b) {
  if (!c.history) return -1;
  const int64_t s = c.slot ? (int64_t)__ldg(c.slot + b) : b;
  return s >= 0 && s < c.state_rows ? s : -1;
}

__device__ __forceinline__ RowConstraints row_constraints(const ConstrainArgs& c, int64_t b) {
  RowConstraints r;
  r.mask = nullptr;
  r.touched = nullptr;
  r.history = nullptr;
  r.bias = nullptr;
  if (c.mask) {
    const int64_t m = c.mask_row ? (int64_t)__ldg(c.mask_row + b) : b;
    if (m >= 0 && m < c.mask_rows) r.mask = c.mask + m * c.mask_ld_bytes;
  }
  const int64_t s = state_row_of(c, b);
  if (s >= 0) {
    r.touched = c.touched + s * (c.state_ld / 8);
    r.history = c.history + s * c.state_ld;
    if (c.bias) r.bias = c.bias + s * c.state_ld;
  }
  r.pen = row_penalties(c, b);
  return r;
}

// A row's bits alone, and where its state row starts (elements; -1: none).
struct RowBits {
  const uint8_t* mask;
  const uint8_t* touched;
  int64_t state;
};

__device__ __forceinline__ RowBits row_bits(const ConstrainArgs& c, int64_t b) {
  RowBits r{nullptr, nullptr, -1};
  if (c.mask) {
    const int64_t m = c.mask_row ? (int64_t)__ldg(c.mask_row + b) : b;
    if (m >= 0 && m < c.mask_rows) r.mask = c.mask + m * c.mask_ld_bytes;
  }
  const int64_t s = state_row_of(c, b);
  if (s >= 0) {
    r.state = s * c.state_ld;
    r.touched = c.touched + r.state / 8;
  }
  return r;
}

// One logit of a row.
template <int DT>
__device__ __forceinline__ float logit_at(const char* row, int32_t v) {
  if constexpr (DT == 0) {
    return __ldcg(reinterpret_cast<const float*>(row) + v);
  } else {
    return half_to_f32<DT>(__ldcg(reinterpret_cast<const unsigned short*>(row) + v));
  }
}

// Logit x of a touched token with history word h and bias `bias`.
__device__ __forceinline__ float penalised(float x, uint32_t h, float bias,
                                           const RowPenalties& r) {
  if (x == -INFINITY) return x;
  float y = __fadd_rn(x, bias);
  if (h != 0u) y = y > 0.0f ? __fdiv_rn(y, r.rep) : __fmul_rn(y, r.rep);
  const uint32_t c = h & 0x7FFFFFFFu;
  if (c != 0u) y = __fsub_rn(__fsub_rn(y, __fmul_rn(r.freq, __uint2float_rn(c))), r.pres);
  return y;
}

// ---------------------------------------------------------------------------
// Units in shared memory. The samplers hold rows as 16-byte units of EPU
// elements: binary32 bits, or raw 16-bit values. Before a sampler looks at its
// units, every masked element becomes -inf, and every touched one
//   - its constrained value, in binary32 units;
//   - in 16-bit units of a sampled row, that value rounded UP to the type: the
//     pruning tests only need a bound from above, and the exact pass forms the
//     value again from the logit (exact_touched);
//   - in 16-bit units of a greedy row, -inf, after the binary32 value has been
//     offered to the running best itself.
// ---------------------------------------------------------------------------

// The value of `y` rounded up to the 16-bit type (NaN, which is never drawn: -inf).
template <int DT>
__device__ __forceinline__ uint32_t bound_bits(float y) {
  constexpr uint32_t ninf = DT == 1 ? 0xFF80u : 0xFC00u;
  if (y != y) return ninf;
  if constexpr (DT == 1) {
    const __nv_bfloat16 h = __float2bfloat16_ru(y);
    return *reinterpret_cast<const unsigned short*>(&h);
  } else {
    const __half h = __float2half_ru(y);
    return *reinterpret_cast<const unsigned short*>(&h);
  }
}

__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint32_t v;
  asm volatile("{\n\t.reg .u16 t;\n\tld.shared.u16 t, [%1];\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ void sts_u16(uint32_t a, uint32_t v) {
  asm volatile("{\n\t.reg .u16 t;\n\tcvt.u16.u32 t, %1;\n\tst.shared.u16 [%0], t;\n\t}" ::"r"(a), "r"(v) : "memory");
}

__device__ __forceinline__ float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ void sts_f32(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// The touched and allowed elements of a thread's units u0, u0 + ustride, ... (at
// shared addresses a0, a0 + 16 * STRIDE, ...): bit 8 * k + e of `todo` stands
// for element e of the k-th unit. Eight elements' state words are fetched at a
// time (of 2, 4, 6 and 8 the fastest: 24.8 us at B = 64, V = 151936 bf16, 4 and
// 2 taking 27.0 and 29.4).
template <int DT, bool F32BITS, int EPU, int STRIDE>
__device__ __forceinline__ void apply_touched(uint32_t a0, int32_t u0, int32_t ustride,
                                              uint64_t todo, const RowConstraints& r,
                                              bool sampled, float& bs, int32_t& bi) {
  constexpr int N = 8;
  while (todo != 0ull) {
    uint32_t at[N], h[N];
    int32_t v[N];
    float b[N];
    bool on[N];
#pragma unroll
    for (int q = 0; q < N; ++q) {
      on[q] = todo != 0ull;
      const int j = on[q] ? __ffsll((long long)todo) - 1 : 0;
      todo &= todo - 1ull;  // 0 stays 0
      const int k = j >> 3, e = j & 7;
      v[q] = (u0 + k * ustride) * EPU + e;
      at[q] = a0 + (uint32_t)(k * STRIDE) * 16u + (uint32_t)e * (F32BITS ? 4u : 2u);
      h[q] = on[q] ? __ldcg(r.history + v[q]) : 0u;
      b[q] = on[q] && r.bias ? __ldcg(r.bias + v[q]) : 0.0f;
    }
#pragma unroll
    for (int q = 0; q < N; ++q) {
      if (!on[q]) continue;
      if constexpr (F32BITS) {
        sts_f32(at[q], penalised(lds_f32(at[q]), h[q], b[q], r.pen));
      } else {
        const float y = penalised(half_to_f32<DT>(lds_u16(at[q])), h[q], b[q], r.pen);
        if (sampled) {
          sts_u16(at[q], bound_bits<DT>(y));
        } else {
          take_better(y, v[q], bs, bi);
          sts_u16(at[q], DT == 1 ? 0xFF80u : 0xFC00u);
        }
      }
    }
  }
}

// A unit with the elements whose bit in `allowed` is clear set to -inf.
template <int DT, bool F32BITS>
__device__ __forceinline__ uint4 masked_unit(uint4 r, uint32_t allowed) {
  uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32BITS) {
      if (!((allowed >> i) & 1u)) w[i] = 0xFF800000u;
    } else {
      constexpr uint32_t ninf = DT == 1 ? 0xFF80u : 0xFC00u;
      // the two bits, 16 apart, widened to halves
      const uint32_t two = (allowed >> (2 * i)) & 3u;
      const uint32_t keep = ((two | two << 15) & 0x10001u) * 0xFFFFu;
      w[i] = (w[i] & keep) | ((ninf * 0x10001u) & ~keep);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The constrained value of a touched element of a 16-bit row, from its logit.
template <int DT>
__device__ __forceinline__ float exact_touched(const char* row, int32_t v,
                                               const RowConstraints& r) {
  return penalised(logit_at<DT>(row, v), __ldcg(r.history + v),
                   r.bias ? __ldcg(r.bias + v) : 0.0f, r.pen);
}

// The value of element v of a 16-bit row whose place holds `x`: a bound, if it
// is touched.
template <int DT>
__device__ __forceinline__ float exact_value(int32_t v, float x, const char* row,
                                             const RowConstraints& r) {
  if (r.touched && (((uint32_t)__ldcg(r.touched + (v >> 3)) >> (v & 7)) & 1u))
    return exact_touched<DT>(row, v, r);
  return x;
}

// The values of group g (elements 4 g .. 4 g + 3) of a 16-bit row whose touched
// elements hold bounds: those get their exact values.
template <int DT>
__device__ __forceinline__ void exact_group(uint32_t g, float (&x)[4], const char* row,
                                            const RowConstraints& r) {
  if (!r.touched) return;
  const uint32_t bits = (uint32_t)__ldcg(r.touched + (g >> 1)) >> (4u * (g & 1u));
#pragma unroll
  for (int t = 0; t < 4; ++t)
    if (((bits >> t) & 1u) && x[t] > -INFINITY)
      x[t] = exact_touched<DT>(row, (int32_t)(4u * g) + t, r);
}

// The N bits (N = 4 or 8) of a bit row that belong to the unit starting at
// element e0, a multiple of N.
template <int N>
__device__ __forceinline__ uint32_t unit_bits(const uint8_t* bits, int32_t e0) {
  const uint32_t v = __ldcg(bits + (e0 >> 3));
  return N == 8 ? v : (v >> (e0 & 4)) & 0xFu;
}

// Logit x of element v, constrained: the element-by-element form.
__device__ __forceinline__ float constrained_logit(float x, int32_t v, const RowConstraints& r) {
  if (r.touched && (__ldcg(r.touched + (v >> 3)) >> (v & 7) & 1u))
    x = penalised(x, __ldcg(r.history + v), r.bias ? __ldcg(r.bias + v) : 0.0f, r.pen);
  if (r.mask && !(__ldcg(r.mask + (v >> 3)) >> (v & 7) & 1u)) x = -INFINITY;
  return x;
}

}  // namespace gsample
