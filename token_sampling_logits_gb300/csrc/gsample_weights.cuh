// Softmax weights in fixed point and the description of a row's filter set:
// shared by the draw from given random numbers and the verification of drafts.
//
// Weights. A row's weights are e_i = 2^(x_i r - C), r = log2(e) / T, with C the
// multiple of 1/256 nearest to M r (M the row's largest logit): one factor
// away from exp((x_i - M) / T) for the whole row, which a draw does not see.
// They are integers in units of 2^-F, so sums are exact, the same in any order
// and for any split of the row, and cumulative sums compare exactly with a
// target. 2^y is the table-driven form of P. T. P. Tang, "Table-driven
// implementation of the exponential function in IEEE floating-point
// arithmetic" (ACM TOMS 15(2), 1989), with a table of 256 steps and a cubic
// for the rest: y = x r is kept as an unevaluated pair of binary32, the cubic
// as 40 fraction bits. A weight is off by at most about 2^-39 of itself plus
// half a unit 2^-F, and the errors of different elements are independent: with
// binary32 weights a draw among 152K equal tokens would name a neighbour of
// the right index in a few of a hundred rows.
#pragma once

#include <cstdint>

#include "gsample_device.cuh"

namespace gsample {

constexpr float kLog2eF = 1.4426950408889634f;
constexpr double kLog2e64 = 1.4426950408889634074;
constexpr double kLn2 = 0.69314718055994530942;

// 2^(i/16) and 2^(i/256) in units of 2^-63: their products are the table.
__constant__ unsigned long long kExp2Coarse[16] = {
    0x8000000000000000ull, 0x85AAC367CC487B15ull, 0x8B95C1E3EA8BD6E7ull, 0x91C3D373AB11C336ull,
    0x9837F0518DB8A96Full, 0x9EF5326091A111AEull, 0xA5FED6A9B15138EAull, 0xAD583EEA42A14AC6ull,
    0xB504F333F9DE6484ull, 0xBD08A39F580C36BFull, 0xC5672A115506DADDull, 0xCE248C151F8480E4ull,
    0xD744FCCAD69D6AF4ull, 0xE0CCDEEC2A94E111ull, 0xEAC0C6E7DD24392Full, 0xF5257D152486CC2Cull};
__constant__ unsigned long long kExp2Fine[16] = {
    0x8000000000000000ull, 0x8058D7D2D5E5F6B1ull, 0x80B1ED4FD999AB6Cull, 0x810B40A1D81406D4ull,
    0x8164D1F3BC030773ull, 0x81BEA1708DDE6056ull, 0x8218AF4373FC25ECull, 0x8272FB97B2A5894Cull,
    0x82CD8698AC2BA1D7ull, 0x83285071E0FC4547ull, 0x8383594EEFB6EE37ull, 0x83DEA15B9541B132ull,
    0x843A28C3ACDE4046ull, 0x8495EFB3303EFD30ull, 0x84F1F656379C1A29ull, 0x854E3CD8F9C8C95Dull};
constexpr int kExp2Entries = 256;

// Entry j of the table: 2^(j/256) in units of 2^-62.
__device__ __forceinline__ unsigned long long exp2_entry(int j) {
  return __umul64hi(kExp2Coarse[j >> 4], kExp2Fine[j & 15]);
}

// Constants of a row's weights.
struct WeightRow {
  float rh, rl;  // log2(e) / T as a pair
  float base;    // subtracted from the logit first (0, or M where x r is too large to be split finely)
  int32_t bias;  // what the bits of y + 49152 are for y = C, in steps of 1/256
  int32_t unit;  // 62 - F
  bool shift;
};

// T > 0 and M finite. Temperatures below 2^-126 count as that. y is split on
// the grid of 1/256 while it stays below 2^14; its rounding error (2^-48 of
// it) asks for a smaller one.
__device__ __forceinline__ WeightRow weight_row(float M, float T, int fraction_bits) {
  constexpr int kMagicBits = 0x47400000;  // 49152.0f: adding it rounds to 1/256
  const double r = kLog2e64 / (double)fmaxf(T, 1.17549435e-38f);
  WeightRow w;
  w.rh = (float)r;
  w.rl = (float)(r - (double)w.rh);
  const double c = (double)M * r;
  w.shift = !(fabs(c) <= 512.0);
  w.base = w.shift ? M : 0.0f;
  w.bias = kMagicBits + (w.shift ? 0 : __double2int_rn(c * 256.0));
  w.unit = 62 - fraction_bits;
  return w;
}

// The weight of logit x <= M (-inf and NaN: 0) in units of 2^-F.
// `table` is the shared-memory address of the 256 entries.
__device__ __forceinline__ unsigned long long weight_of(float x, const WeightRow& w,
                                                        uint32_t table) {
  float d = x, dl = 0.0f;
  if (w.shift) {  // x - M as an exact pair
    d = x - w.base;
    const float b = d - x;
    dl = (x - (d - b)) + (-w.base - b);
  }
  // y = d r as the pair (p, e)
  float p = d * w.rh;
  float e = fmaf(d, w.rl, fmaf(d, w.rh, -p));
  if (w.shift) e = fmaf(dl, w.rh, e);
  // p = k / 256 + g; an element far below (-inf, NaN) ends with a very negative k
  p = fmaxf(p, -16000.0f);
  const float kf = p + 49152.0f;
  const int32_t k = __float_as_int(kf) - w.bias;
  const int32_t s = w.unit - (k >> 8);
  if (s > 63) return 0ull;
  const float g0 = p - (kf - 49152.0f);
  const float g = g0 + e;
  const float ge = e - (g - g0);
  // 2^g - 1 = a + t, a = g ln 2 to 24 bits
  constexpr float kLn2h = 0.693147182464599609375f, kLn2l = (float)(kLn2 - 0.693147182464599609375);
  const float a = g * kLn2h;
  float t = fmaf(ge, kLn2h, fmaf(g, kLn2l, fmaf(g, kLn2h, -a)));
  t = fmaf(a * a, fmaf(a, 1.0f / 6.0f, 0.5f), t);
  // a + t in units of 2^-40: a to 2^-31, what that leaves joins t
  constexpr float kA = 1.5f / 256.0f, kT = 1.5f / 131072.0f;
  const float va = a + kA;
  const float vt = t + (a - (va - kA)) + kT;
  const int32_t q = ((__float_as_int(va) - __float_as_int(kA)) << 9) +
                    (__float_as_int(vt) - __float_as_int(kT));
  const uint2 tab = lds64(table + (uint32_t)(k & 255) * 8u);
  const long long base = (long long)(((unsigned long long)tab.y << 32) | tab.x);
  const long long v = base + (((long long)(int32_t)tab.y * (long long)q) >> 8);
  return (((unsigned long long)v >> (s - 1)) + 1ull) >> 1;
}

// u in [0, 1) (smaller, or NaN: 0; larger: the largest below 1) in units of 2^-64.
__device__ __forceinline__ unsigned long long fraction_of(float u) {
  if (!(u > 0.0f)) return 0ull;
  u = fminf(u, 0.999999940395355224609375f);
  return (unsigned long long)__float2ull_rz(u * 18446744073709551616.0f);
}

// ceil(f * s / 2^64)
__device__ __forceinline__ unsigned long long ceil_part(unsigned long long f,
                                                        unsigned long long s) {
  return __umul64hi(f, s) + (f * s != 0ull ? 1ull : 0ull);
}

// What a row draws from. kSet: the elements whose ordered key is above `key`,
// and those equal to it up to index `last`, with weights as above and their sum.
enum RowKind : int32_t { kNothing = 0, kOne = 1, kSet = 2 };
struct RowSet {
  unsigned long long sum;
  float M;
  uint32_t key;
  int32_t last;  // kOne: the index
  int32_t kind;
  int32_t accepted;  // the draft of this row passed its test
  int32_t request;
};
static_assert(sizeof(RowSet) == 32, "32 bytes a row of the verification's workspace");

}  // namespace gsample
