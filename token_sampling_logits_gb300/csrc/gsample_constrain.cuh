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
// State and mask words are read once a launch, through L2 only (ld.cg): a state
// row is often rewritten by the kernel just before on the stream.
#pragma once

#include <cstdint>

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

// One batch row's view of them; a null pointer means "none for this row".
struct RowConstraints {
  const uint8_t* mask;
  const uint8_t* touched;
  const uint32_t* history;
  const float* bias;
  float rep, freq, pres;
};

__device__ __forceinline__ RowConstraints row_constraints(const ConstrainArgs& c, int64_t b) {
  RowConstraints r;
  r.mask = nullptr;
  r.touched = nullptr;
  r.history = nullptr;
  r.bias = nullptr;
  r.rep = 1.0f;
  r.freq = 0.0f;
  r.pres = 0.0f;
  if (c.mask) {
    const int64_t m = c.mask_row ? (int64_t)__ldg(c.mask_row + b) : b;
    if (m >= 0 && m < c.mask_rows) r.mask = c.mask + m * c.mask_ld_bytes;
  }
  if (c.history) {
    const int64_t s = c.slot ? (int64_t)__ldg(c.slot + b) : b;
    if (s >= 0 && s < c.state_rows) {
      r.touched = c.touched + s * (c.state_ld / 8);
      r.history = c.history + s * c.state_ld;
      if (c.bias) r.bias = c.bias + s * c.state_ld;
    }
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
  }
  return r;
}

// Logit x of a touched token with history word h and bias `bias`.
__device__ __forceinline__ float penalised(float x, uint32_t h, float bias,
                                           const RowConstraints& r) {
  if (x == -INFINITY) return x;
  float y = __fadd_rn(x, bias);
  if (h != 0u) y = y > 0.0f ? __fdiv_rn(y, r.rep) : __fmul_rn(y, r.rep);
  const uint32_t c = h & 0x7FFFFFFFu;
  if (c != 0u) y = __fsub_rn(__fsub_rn(y, __fmul_rn(r.freq, __uint2float_rn(c))), r.pres);
  return y;
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
    x = penalised(x, __ldcg(r.history + v), r.bias ? __ldcg(r.bias + v) : 0.0f, r);
  if (r.mask && !(__ldcg(r.mask + (v >> 3)) >> (v & 7) & 1u)) x = -INFINITY;
  return x;
}

}  // namespace gsample
