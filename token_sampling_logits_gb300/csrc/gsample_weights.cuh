// Softmax weights in fixed point and the description of a row's filter set:
// shared by the draw from given random numbers and the verification of drafts.
//
// Weights. A row's weights are e_i = 2^(x_i r - C), r = log2(e) / T, with C the
// multiple of 1/256 nearest to M r (M the row's largest logit): one factor
// away from exp((x_i - M) / T) for the whole row, which a draw does not see.
// They are integers in units of 2^-44, so sums are exact, the same in any order
// and for any split of the row, and cumulative sums compare exactly with a
// target. 2^y is the table-driven form of P. T. P. Tang, "Table-driven
// implementation of the exponential function in IEEE floating-point
// arithmetic" (ACM TOMS 15(2), 1989), with a table of 256 steps and a cubic
// for the rest, all of it on unevaluated pairs of binary32: two elements share
// each instruction (fma.rn.f32x2), where 64-bit integers for the same number
// of bits took 89 instructions an element. A weight is off by at most about
// 2^-39 of itself plus half a unit, and the errors of different elements are
// independent: with binary32 weights a draw among 152K equal tokens would name
// a neighbour of the right index in a few of a hundred rows.
#pragma once

#include <cstdint>

#include "gsample_device.cuh"

namespace gsample {

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

// Entry j of the table: 2^(j/256) as a pair of binary32.
__device__ __forceinline__ float2 exp2_entry(int j) {
  const unsigned long long v = __umul64hi(kExp2Coarse[j >> 4], kExp2Fine[j & 15]);  // 2^-62 units
  const unsigned long long h = (v + (1ull << 38)) >> 39;                            // 2^-23 units
  const long long rest = (long long)(v - (h << 39));
  // (a low half of 0, that of 2^0, would not stand the exponents added below)
  return make_float2((float)(uint32_t)h * 1.1920928955078125e-07f,
                     rest ? (float)rest * 2.16840434497100886801e-19f : 2.8421709430404007e-14f);
}

// Two binary32 numbers that share an instruction.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void split(F2 a, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 sub2(F2 a, F2 b) {
  F2 r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// Constants of a row's weights.
struct WeightRow {
  float rh, rl;  // log2(e) / T as a pair
  float M;
  float lowest;  // logits below this (-inf and NaN too) have weight 0
  float c;       // what is taken off y: the multiple of 1/256 nearest to M r, or 0
  float scale;   // `shift`: a power of two that keeps x - M in range
  int32_t bias;  // the bits of y + 49152 at y = C
  bool shift;    // M is subtracted first: x r is too large to be split finely, or T so
                 // large that `lowest` cannot stand in for -inf
};

constexpr int kMagicK = 0x47400000;           // 49152.0f: adding it rounds y to 1/256
constexpr float kMagicH = 2.5f;               // rounds a weight in [0, 1.5) to 2^-22
constexpr float kMagicL = 1.5f / 2097152.0f;  // rounds what that leaves to 2^-44
constexpr float kLowestLogit = -3.402823466e38f;

// T > 0. Temperatures below 2^-126 count as that.
__device__ __forceinline__ void weight_scale(float T, float& scale, float& rh, float& rl) {
  constexpr float kLog2eH = 1.44269502162933349609375f, kLog2eL = 1.9259629911266175e-08f;
  T = fmaxf(T, 1.17549435e-38f);
  scale = T > 1e30f ? 0.25f : 1.0f;
  rh = rl = 0.0f;
  if (T < INFINITY) {
    const float t = T * scale;
    const float q = __fdiv_rn(kLog2eH, t);
    const float l = __fdiv_rn(__fadd_rn(__fmaf_rn(-q, t, kLog2eH), kLog2eL), t);
    rh = __fadd_rn(q, l);
    rl = __fsub_rn(l, __fsub_rn(rh, q));
  }
}

// T > 0 and M finite. `drop` powers of two are taken off the weights (rows of
// more than 2^18 elements).
__device__ __forceinline__ WeightRow weight_row(float M, float T, int drop) {
  WeightRow w;
  weight_scale(T, w.scale, w.rh, w.rl);
  w.M = M;
  const float c = M * w.rh;
  const float lowest = M - 42.0f * fmaxf(T, 1.17549435e-38f);  // 60 powers of two below M
  w.lowest = fmaxf(lowest, kLowestLogit);
  w.shift = !(fabsf(c) <= 512.0f) || !(lowest >= kLowestLogit);
  const int steps = w.shift ? 0 : __float2int_rn(c * 256.0f);
  w.c = (float)steps * 0.00390625f + (float)drop;
  w.bias = kMagicK + steps + drop * 256;
  return w;
}

// The weights of two logits x <= M: 2^-22 (h - the bits of kMagicH) + 2^-44
// (l - the bits of kMagicL). `table` is the shared-memory address of the 256
// entries. Products and differences of one value are formed from its negative
// (n...), which rounds alike.
template <bool SHIFT>
__device__ __forceinline__ void weight_bits(float x0, float x1, const WeightRow& w, uint32_t table,
                                            int32_t (&h)[2], int32_t (&l)[2]) {
  F2 x = f2(fmaxf(x0, w.lowest), fmaxf(x1, w.lowest)), xl = f2(0.0f);
  bool z0 = true, z1 = true;
  if constexpr (SHIFT) {  // x - M as an exact pair
    x = mul2(x, f2(w.scale));
    const F2 m = f2(w.M * w.scale), d = sub2(x, m);
    const F2 b = sub2(d, x);
    xl = sub2(sub2(x, sub2(d, b)), add2(m, b));
    float d0, d1, l0, l1;
    split(d, d0, d1);
    split(xl, l0, l1);
    z0 = x0 >= w.lowest && d0 * w.rh > -64.0f;
    z1 = x1 >= w.lowest && d1 * w.rh > -64.0f;
    x = f2(z0 ? d0 : 0.0f, z1 ? d1 : 0.0f);
    xl = f2(z0 ? l0 : 0.0f, z1 ? l1 : 0.0f);
  }
  // y = x r as the pair (p, e)
  const F2 rh = f2(w.rh), np = mul2(x, f2(-w.rh));
  F2 e = fma2(x, f2(w.rl), fma2(x, rh, np));
  if constexpr (SHIFT) e = fma2(xl, rh, e);
  // p = k / 256 + g0; y = k / 256 + g + ge
  const F2 kf = sub2(f2(49152.0f), np);
  const F2 ng0 = add2(np, sub2(kf, f2(49152.0f)));
  const F2 g = sub2(e, ng0);
  const F2 ge = sub2(e, add2(g, ng0));
  // 2^(g + ge) - 1 = a + t, a = g ln 2 to 24 bits
  const F2 ln2h = f2(0.693147182464599609375f);
  const F2 a = mul2(g, ln2h), na = mul2(g, f2(-0.693147182464599609375f));
  F2 t = fma2(ge, ln2h, fma2(g, f2(-1.90465429995776793e-09f), fma2(g, ln2h, na)));
  t = fma2(mul2(a, a), fma2(a, f2(1.0f / 6.0f), f2(0.5f)), t);
  float kf0, kf1;
  split(kf, kf0, kf1);
  const int32_t k0 = __float_as_int(kf0) - w.bias, k1 = __float_as_int(kf1) - w.bias;
  const uint2 t0 = lds64(table + ((uint32_t)k0 & 255u) * 8u);
  const uint2 t1 = lds64(table + ((uint32_t)k1 & 255u) * 8u);
  const int32_t n0 = (k0 >> 8) << 23, n1 = (k1 >> 8) << 23;  // added to the exponents
  const F2 th = f2(__int_as_float((int32_t)t0.x + n0), __int_as_float((int32_t)t1.x + n1));
  const F2 tl = f2(__int_as_float((int32_t)t0.y + n0), __int_as_float((int32_t)t1.y + n1));
  // (th + tl) (1 + a + t) = v + lo
  const F2 nu = mul2(th, na);
  F2 lo = add2(fma2(tl, a, fma2(th, t, fma2(th, a, nu))), tl);
  const F2 v = sub2(th, nu);
  lo = sub2(lo, add2(nu, sub2(v, th)));
  const F2 vh = add2(add2(v, lo), f2(kMagicH));
  const F2 vl = add2(add2(sub2(v, sub2(vh, f2(kMagicH))), lo), f2(kMagicL));
  float h0, h1, l0, l1;
  split(vh, h0, h1);
  split(vl, l0, l1);
  h[0] = __float_as_int(z0 ? h0 : kMagicH);
  h[1] = __float_as_int(z1 ? h1 : kMagicH);
  l[0] = __float_as_int(z0 ? l0 : kMagicL);
  l[1] = __float_as_int(z1 ? l1 : kMagicL);
}

constexpr int32_t kBitsH = 0x40200000;  // 2.5f
constexpr int32_t kBitsL = 0x35400000;  // 1.5 * 2^-21

// The weights of two logits x <= M in units of 2^-44. (Out of line: where few
// elements are weighed the instructions that are fetched count for more.)
static __device__ __noinline__ void weights_of(float x0, float x1, const WeightRow& w, uint32_t table,
                                           unsigned long long (&v)[2]) {
  int32_t h[2], l[2];
  if (w.shift)
    weight_bits<true>(x0, x1, w, table, h, l);
  else
    weight_bits<false>(x0, x1, w, table, h, l);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    v[i] = (unsigned long long)(((long long)(h[i] - kBitsH) << 22) + (long long)(l[i] - kBitsL));
}
__device__ __forceinline__ unsigned long long weight_of(float x, const WeightRow& w,
                                                        uint32_t table) {
  unsigned long long v[2];
  weights_of(x, x, w, table, v);
  return v[0];
}

// A sum of weights of a thread's elements: the two parts apart, in 32 bits,
// joined before either can run over (at most 256 pairs).
struct WeightSum {
  uint32_t h = 0u, l = 0u;
  __device__ __forceinline__ void add(const int32_t (&a)[2], const int32_t (&b)[2]) {
    h += (uint32_t)a[0] + (uint32_t)a[1];
    l += (uint32_t)b[0] + (uint32_t)b[1];
  }
  // `n`: elements added since the last call
  __device__ __forceinline__ unsigned long long take(uint32_t n) {
    const uint32_t sh = h - n * (uint32_t)kBitsH;
    const int32_t sl = (int32_t)(l - n * (uint32_t)kBitsL);
    h = l = 0u;
    return ((unsigned long long)sh << 22) + (unsigned long long)(long long)sl;
  }
};

// v > 0 as 2^(n / 256) times 1 + r, |r| < 2^-9, r as a pair.
struct LogParts {
  int32_t n;
  float rh, rl;
};
__device__ __forceinline__ LogParts log_parts(unsigned long long v, uint32_t table) {
  const int up = __clzll((long long)v);
  v <<= up;  // 2^-63 units of a number in [1, 2)
  const uint32_t top = (uint32_t)(v >> 40);  // 24 bits
  const float mh = (float)top * 1.1920928955078125e-07f;
  const float ml = (float)(uint32_t)((v >> 8) & 0xFFFFFFFFull) * 2.7755575615628914e-17f;
  const int k = min(255, __float2int_rn(256.0f * __log2f(mh)));
  const uint2 t = lds64(table + (uint32_t)k * 8u);
  const float th = __uint_as_float(t.x), tl = __uint_as_float(t.y);
  const float d = __fadd_rn(__fsub_rn(mh, th), 0.0f);  // exact
  const float e = __fsub_rn(ml, tl);
  const float rh = __fdividef(__fadd_rn(d, e), th);
  // d + e - rh (th + tl), over th
  float rest = __fmaf_rn(-rh, th, d);
  rest = __fadd_rn(rest, e);
  rest = __fmaf_rn(-rh, tl, rest);
  return LogParts{(63 - up) * 256 + k, rh, __fdividef(rest, th)};
}

// ln(w / s), 0 < w <= s, rounded once (and off by at most 2^-40 before): by the
// steps of the table, the rest of each number by its series (Tang, as above).
__device__ __forceinline__ float log_ratio(unsigned long long w, unsigned long long s,
                                           uint32_t table) {
  if (w >= s) return 0.0f;
  const LogParts a = log_parts(w, table), b = log_parts(s, table);
  auto series = [](const LogParts& p) {  // ln(1 + r) - rh
    const float q = p.rh * p.rh;
    return fmaf(q, fmaf(p.rh, fmaf(p.rh, -0.25f, 1.0f / 3.0f), -0.5f), p.rl * (1.0f - p.rh));
  };
  // (n_a - n_b) ln2 / 256 as a pair, then the differences of the series
  constexpr float ch = 0.0027076061815023422f, cl = -7.4400558592100308e-12f;
  const float n = (float)(a.n - b.n);
  const float p = n * ch, pl = fmaf(n, cl, fmaf(n, ch, -p));
  const float d = a.rh - b.rh, db = d - a.rh;
  const float dl = (a.rh - (d - db)) + (-b.rh - db);
  const float sum = p + d, sb = sum - p;
  const float sl = (p - (sum - sb)) + (d - sb);
  return sum + (sl + (pl + (dl + (series(a) - series(b)))));
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
enum RowKind : int32_t { kNothing = 0, kOne = 1, kSet = 2, kOpen = 3 };
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
