// The draw from a row's top-k / top-p / min-p set with the caller's random
// number, and the verification of speculative drafts by the same sets.
//
// The set K of a row is a prefix of its candidates (logits that are neither
// NaN nor -inf) in the order (logit descending, index ascending): it ends at
// the first of top_k elements, of the shortest prefix whose softmax mass
// reaches top_p, and of the elements of at least min_p times the largest
// probability. The draw is the inverse CDF over K in index order.
//
// Layout: one thread-block cluster per row, each CTA a slice of the row, each
// warp a run of it, so that ranks, warps, lanes and units (16 bytes) follow the
// index order. One sweep reads the row: its maximum, each unit's own maximum
// (sixteen bits, in shared memory), and for rows whose mass is asked for the sum
// of their weights in binary32. Then a row takes the first of these ways that
// settles it:
//   - one element only (greedy, +inf, nothing): the lowest index of the maximum;
//   - short sets: the elements within 12 powers of two of the maximum (a few
//     dozen of a language model's row; for a top_k alone, about as many as it
//     asks for) are listed from the units that hold them, in index order, and
//     sent to rank 0, which finds K's end with exact weights and draws. What is
//     not listed of the mass (top_p) is the binary32 sum, with a bound on its
//     error: the row is not settled when the bound leaves K's end open, a list
//     runs over or K reaches past it. Without a filter the same sums tell the warp
//     whose run u falls in, and there the unit and the element;
//   - long sets: a histogram of the logits in 4096 equal steps brackets K's
//     end; one sweep forms the exact weights of all, sums those above the
//     bracket and lists those in it; rank 0 finds K's end; the draw is by the
//     warps' sums;
//   - the rest (very many logits in the bracket, or an estimate that missed): a
//     radix select over order-preserving keys with counts and exact masses, eight
//     bits a level.
// All sums but the bounded ones are integers (gsample_weights.cuh), so the
// result does not depend on the way taken, the order of any atomic or the
// split of the row. The only waits are hardware barriers.
//
// Measured at V = 151936 bf16 (the 77.8 MB of 256 rows take 11.5 us at the copy's
// rate): 256 rows with mixed filters 48 to 62 us, 92 when one of them is a long
// set; without filters 50 us; 64 rows whose nuclei hold 10^4 to 10^5 tokens 91 us.
// A short row's time is the sweep (20 us with weights, 10 without), then a chain
// of small steps between barriers (12 us), whose instructions come from L2 as
// often as not. Holding the slice in shared memory instead (76 KB a CTA, 4 CTAs a
// row) took 73 us for the sweep and list; every weight exact 104 us.
#pragma once

#include <cooperative_groups.h>

#include <climits>
#include <cstddef>
#include <type_traits>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gsample_internal.h"
#include "gsample_slice.cuh"
#include "gsample_weights.cuh"

namespace cg = cooperative_groups;

namespace gsample {
namespace {

using namespace slice;

constexpr int kDrawThreads = 512;
constexpr int kDrawWarps = kDrawThreads / 32;
constexpr int kDrawMaxCluster = 16;
constexpr int kMaxSegments = kDrawMaxCluster * kDrawWarps;
constexpr int kWarpList = 64;                 // entries of a warp's list
constexpr int kCtaList = kWarpList * kDrawWarps;
constexpr int kRowList = 1280;                // entries of a row's list, at rank 0
constexpr int kLandList = 768;
constexpr int kListBins = 512;
constexpr int kBins = 4096;                   // steps of the histogram
constexpr int64_t kOpenIndex = -2;            // out_idx of a row left to the second launch

using u64 = unsigned long long;

template <int DT>
__device__ __forceinline__ float logit_at(const char* row, int64_t i) {
  if constexpr (DT == 0) {
    return __ldg(reinterpret_cast<const float*>(row) + i);
  } else {
    return half_to_f32<DT>(__ldg(reinterpret_cast<const unsigned short*>(row) + i));
  }
}

// Order-preserving keys in the bits that the logit's dtype can set.
template <int DT>
struct KeyBits {
  static constexpr int kZB = DT == 1 ? 16 : (DT == 2 ? 13 : 0);
};

template <int DT>
__device__ __forceinline__ uint32_t key_of_short(uint32_t s) {
  constexpr int ZB = KeyBits<DT>::kZB;
  if constexpr (ZB == 0) {
    return s;
  } else {
    const uint32_t k = s << ZB;
    return (k & 0x80000000u) ? k : (k | ((1u << ZB) - 1u));
  }
}

__device__ __forceinline__ float logit_of_key(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

struct alignas(16) Ranked {  // an element of the bin that K ends in
  u64 w;
  uint32_t key, idx;
};

struct alignas(16) DrawShared {
  float2 table[kExp2Entries];
  u64 sums[2][kMaxSegments];      // the warps' sums of the whole cluster (two buffers)
  float wmax[kMaxSegments];       // their maxima; then, at rank 0, offsets of their lists
  unsigned count[kMaxSegments];   // at rank 0: the lengths of their lists
  unsigned landed_at[kMaxSegments];  // and where they landed
  unsigned landed_n;
  unsigned near[256], near_all[256];  // units near the maximum, of this CTA and of the row
  union {
    alignas(16) struct {
      unsigned hist[kBins];   // of this CTA; read sixteen bytes at a time
      unsigned steps[kBins];  // of the row
    };
    struct {
      uint2 list[kRowList];  // logit bits and index
      union {
        struct {
          u64 mass[kListBins];
          unsigned count[kListBins];
        } bin;
        Ranked last[kRowList];
        uint2 landed[kLandList];  // as they come from the cluster's warps
      };
    } row;
    struct {
      u64 mass[2][256];  // a level of the radix select (two buffers)
      unsigned count[2][256];
    } digit;
  };
  uint2 own[kCtaList];  // this CTA's lists
  u64 scan_m[kDrawWarps];
  float scan_f[kDrawWarps];
  unsigned scan_c[kDrawWarps];
  int sel[8];
  unsigned above_c, all_c;
  u64 above_m, all_m;
  u64 tail, tail_err, m_lo, m_hi;  // at rank 0
  double floor_step;     // T ln(min_p)
  int32_t found;         // written by the CTA that finds an index
  int32_t request;
  unsigned own_n;
  // K's end, written by rank 0
  int32_t settled;
  uint32_t key;
  int32_t last;
  u64 sum;
};

static_assert(offsetof(DrawShared, hist) % 16 == 0, "the histogram is read as uint4");

// Cluster barriers. Not the .aligned forms, which are undefined where the lanes of
// a warp have not met again after a branch of their own.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void cluster_barrier() {
  cluster_arrive();
  cluster_wait();
}

// The address of this CTA's shared variable in CTA `rank` of the cluster.
template <typename T>
__device__ __forceinline__ T* peer(T* p, int rank) {
  return cg::this_cluster().map_shared_rank(p, rank);
}

// One row's work within its cluster: the slice of this CTA and how to read it.
template <int DT, bool VEC>
struct RowCtx {
  using C = HCfg<DT, VEC>;
  static constexpr int EPU = C::kEPU, kDT = DT;
  static constexpr bool kVec = VEC;
  static constexpr bool kHalfMaxima = VEC && DT == 2;  // unit maxima as f16, else as bf16
  static constexpr int kFlush = 256 / EPU;  // units between joins of a WeightSum
  const char* row;
  int32_t V, u_lo, u_hi;
  int rank, nrank, warp, lane;
  int32_t w_lo, w_hi;  // units of this warp

  __device__ __forceinline__ void place(const DrawParams& p, int64_t b) {
    row = p.logits + b * p.ld_bytes;
    V = p.V;
    u_lo = min(p.units_per_row, rank * p.units_per_cta);
    u_hi = min(p.units_per_row, u_lo + p.units_per_cta);
    run_of(warp, w_lo, w_hi);
  }

  // A warp's run is a multiple of eight units, but for the last.
  static __device__ __forceinline__ int32_t run_length(int32_t n) {
    return ((n + kDrawWarps - 1) / kDrawWarps + 7) / 8 * 8;
  }
  __device__ __forceinline__ void run_of(int w, int32_t& lo, int32_t& hi) const {
    const int32_t n = u_hi - u_lo, per = run_length(n);
    lo = u_lo + min(n, w * per);
    hi = u_lo + min(n, (w + 1) * per);
  }

  // The warp that holds element i of the row, counted over the cluster.
  __device__ __forceinline__ int segment_of(int32_t i, int32_t units, int32_t per_cta) const {
    const int32_t u = i / EPU, q = u / per_cta;
    return q * kDrawWarps + (u - q * per_cta) / run_length(min(per_cta, units - q * per_cta));
  }

  // The warp that holds element i of this CTA's slice.
  __device__ __forceinline__ int warp_of(int32_t i) const {
    return (i / EPU - u_lo) / run_length(u_hi - u_lo);
  }

  // The logits are read once from memory, and where a row is read again, from L2.
  __device__ __forceinline__ uint4 unit(int32_t u) const {
    if constexpr (VEC) {
      if ((u + 1) * EPU <= V) {
        uint4 v;
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(row + (size_t)u * 16));
        return v;
      }
    }
    return load_unit<DT, VEC>(row, u, V, 0ull);
  }

  static __device__ __forceinline__ uint4 no_unit() {  // all -inf
    const uint32_t n = C::kF32Bits ? 0xFF800000u : DT == 1 ? 0xFF80FF80u : 0xFC00FC00u;
    return make_uint4(n, n, n, n);
  }

  // A unit's largest element, rounded up to sixteen bits; and what it is at most.
  static __device__ __forceinline__ uint32_t short_of(float x) {
    if constexpr (kHalfMaxima) {
      return __half_as_ushort(__float2half_ru(x));
    } else {
      const uint32_t b = __float_as_uint(x);
      return (b & 0x80000000u ? b : b + 0xFFFFu) >> 16;
    }
  }
  static __device__ __forceinline__ float of_short(uint32_t s) {
    return half_to_f32<kHalfMaxima ? 2 : 1>(s);
  }
  // What it is at least: the same where the logits have sixteen bits, else the next
  // number down.
  static __device__ __forceinline__ float at_least(uint32_t s) {
    if constexpr (!C::kF32Bits) return of_short(s);
    return of_short(s == 0u ? 0x8001u : s & 0x8000u ? s + 1u : s - 1u);
  }

  static __device__ __forceinline__ float element(const uint4& r, int e) {
    return elt<DT, VEC>(r, e);
  }

  // The largest element of a unit (NaN only where all are).
  static __device__ __forceinline__ float largest(const uint4& r) {
    if constexpr (C::kF32Bits) {
      return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)),
                   fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
    } else {
      return largest_short<DT>(r);
    }
  }
  // The same of eight 16-bit numbers.
  template <int D>
  static __device__ __forceinline__ float largest_short(const uint4& r) {
    {
      uint32_t m;
      if constexpr (D == 1)
        asm("{.reg .b32 a, b;\n max.bf16x2 a, %1, %2;\n max.bf16x2 b, %3, %4;\n max.bf16x2 %0, a, b;}"
            : "=r"(m) : "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w));
      else
        asm("{.reg .b32 a, b;\n max.f16x2 a, %1, %2;\n max.f16x2 b, %3, %4;\n max.f16x2 %0, a, b;}"
            : "=r"(m) : "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w));
      return fmaxf(half_to_f32<D>(m & 0xFFFFu), half_to_f32<D>(m >> 16));
    }
  }

  // f(x, i) on every element of this thread's units, in index order.
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
    uint4 next = w_lo + lane < w_hi ? unit(w_lo + lane) : no_unit();
    for (int32_t u = w_lo + lane; u < w_hi; u += 32) {
      const uint4 r = next;
      if (u + 32 < w_hi) next = unit(u + 32);
#pragma unroll
      for (int e = 0; e < EPU; ++e) f(element(r, e), u * EPU + e);
    }
  }

  // f(x0, x1, i) on every pair of neighbours; g() after every kFlush units.
  template <typename F, typename G>
  __device__ __forceinline__ void each_pair(F&& f, G&& g) const {
    int n = 0;
    uint4 next = w_lo + lane < w_hi ? unit(w_lo + lane) : no_unit();
    for (int32_t u = w_lo + lane; u < w_hi; u += 32) {
      const uint4 r = next;
      if (u + 32 < w_hi) next = unit(u + 32);
#pragma unroll
      for (int e = 0; e < EPU; e += 2) f(element(r, e), element(r, e + 1), u * EPU + e);
      if (++n == kFlush) {
        g(kFlush * EPU);
        n = 0;
      }
    }
    g(n * EPU);
  }
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The row's sum of v; the warps' sums stay in sh.sums[buf]. `buf` alternates
// between calls: a warp may still read one call's sums while another writes the
// next one's.
template <typename Row>
__device__ __forceinline__ u64 cluster_sum(u64 v, const Row& r, DrawShared& sh, int buf) {
  v = warp_sum(v);
  if (r.lane < r.nrank) *peer(&sh.sums[buf][r.rank * kDrawWarps + r.warp], r.lane) = v;
  cluster_barrier();
  u64 all = 0ull;
  for (int q = r.lane; q < r.nrank * kDrawWarps; q += 32) all += sh.sums[buf][q];
  return warp_sum(all);
}

// Inclusive scan over the CTA of one count and one mass a thread.
__device__ __forceinline__ void cta_scan(unsigned& c, u64& m, DrawShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned tc = __shfl_up_sync(0xFFFFFFFFu, c, o);
    const u64 tm = __shfl_up_sync(0xFFFFFFFFu, m, o);
    if (lane >= o) {
      c += tc;
      m += tm;
    }
  }
  if (lane == 31) {
    sh.scan_c[warp] = c;
    sh.scan_m[warp] = m;
  }
  __syncthreads();
  unsigned bc = lane < warp ? sh.scan_c[lane] : 0u;
  u64 bm = lane < warp ? sh.scan_m[lane] : 0ull;
  c += __reduce_add_sync(0xFFFFFFFFu, bc);
  m += warp_sum(bm);
  __syncthreads();
}

// The element at which the cumulative weight passes `target` (< the row's sum),
// after cluster_sum(buf): the CTA that holds it scans the run of the warp that
// held it, a unit a thread, and calls done(index, x, weight) in one thread.
// pair(x0, x1, i, v) gives the weights of elements i and i + 1. Called by the
// whole CTA.
template <typename Row, typename W, typename Done>
__device__ __forceinline__ void find_index(const Row& r, DrawShared& sh, int buf, u64 target,
                                           W&& pair, Done&& done) {
  // which warp: lane l adds the sums of eight of them
  constexpr int kPer = kMaxSegments / 32;
  const int n = r.nrank * kDrawWarps;
  u64 own = 0ull;
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    own += r.lane * kPer + j < n ? sh.sums[buf][r.lane * kPer + j] : 0ull;
  u64 incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (r.lane >= o) incl += t;
  }
  const unsigned past = __ballot_sync(0xFFFFFFFFu, incl > target);
  if (past == 0u) return;  // (target is below the sum)
  const int l = __ffs(past) - 1;
  u64 before = __shfl_sync(0xFFFFFFFFu, incl - own, l);
  int at = l * kPer;
  while (at + 1 < n && before + sh.sums[buf][at] <= target) before += sh.sums[buf][at++];
  if (at / kDrawWarps != r.rank) return;
  u64 left = target - before;
  int32_t lo, hi;
  r.run_of(at % kDrawWarps, lo, hi);
  for (int32_t u0 = lo; u0 < hi; u0 += kDrawThreads) {
    const int32_t u = u0 + (int)threadIdx.x;
    u64 v[Row::EPU];
    u64 sum = 0ull;
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int e = 0; e < Row::EPU; ++e) v[e] = 0ull;
    if (u < hi) {
      q = r.unit(u);
#pragma unroll
      for (int e = 0; e < Row::EPU; e += 2) {
        u64 two[2];
        pair(Row::element(q, e), Row::element(q, e + 1), u * Row::EPU + e, two);
        v[e] = two[0];
        v[e + 1] = two[1];
        sum += two[0] + two[1];
      }
    }
    u64 end = sum;
    unsigned none = 0u;
    cta_scan(none, end, sh);
    u64 c = end - sum;
    if (left >= c && left < end) {
#pragma unroll
      for (int e = 0; e < Row::EPU; ++e) {
        if (left >= c && left < c + v[e]) done(u * Row::EPU + e, Row::element(q, e), v[e]);
        c += v[e];
      }
    }
    // what the units so far hold
    if (threadIdx.x == kDrawThreads - 1) sh.all_m = end;
    __syncthreads();
    const u64 all = sh.all_m;
    __syncthreads();
    if (left < all) return;
    left -= all;
  }
}

// This thread's sum of the weights of the elements from `lowest` up.
template <bool SHIFT, typename Row>
__device__ __forceinline__ u64 sum_from(const Row& r, const WeightRow& w, uint32_t table,
                                        float lowest) {
  u64 sum = 0ull;
  WeightSum part;
  // an element below `lowest` counts as one below w.lowest, which weighs nothing
  const bool all = !SHIFT && lowest <= w.lowest;
  auto join = [&](int n) { sum += part.take((uint32_t)n); };
  if (all) {
    r.each_pair(
        [&](float x0, float x1, int32_t) {
          int32_t h[2], l[2];
          weight_bits<SHIFT>(x0, x1, w, table, h, l);
          part.add(h, l);
        },
        join);
  } else {
    r.each_pair(
        [&](float x0, float x1, int32_t) {
          int32_t h[2], l[2];
          weight_bits<SHIFT>(x0 >= lowest ? x0 : -INFINITY, x1 >= lowest ? x1 : -INFINITY, w, table,
                             h, l);
          part.add(h, l);
        },
        join);
  }
  return sum;
}

// Thread t < 256 holds the totals (c, m) of digit 255 - t. The first digit from
// the top at which the cumulative count reaches k_rem or the cumulative mass
// m_rem (both at least 1), or -1; sh.above_* get the totals above it, sh.all_*
// those of all digits. Called by every thread; ends with a barrier.
__device__ __forceinline__ int find_digit(unsigned c, u64 m, unsigned k_rem, u64 m_rem,
                                          DrawShared& sh) {
  if (threadIdx.x == 0) sh.sel[0] = kDrawThreads;
  unsigned ic = c;
  u64 im = m;
  cta_scan(ic, im, sh);
  if (threadIdx.x < 256 &&
      ((ic - c < k_rem && k_rem <= ic) || (im - m < m_rem && m_rem <= im)))
    atomicMin(&sh.sel[0], (int)threadIdx.x);
  __syncthreads();
  const int at = sh.sel[0];
  if ((int)threadIdx.x == at) {
    sh.above_c = ic - c;
    sh.above_m = im - m;
  }
  if (threadIdx.x == 255) {
    sh.all_c = ic;
    sh.all_m = im;
  }
  __syncthreads();
  return at < 256 ? 255 - at : -1;
}

// The request whose row `b` is, written to sh.request (-1: none; the lowest
// where malformed offsets give several).
__device__ __forceinline__ int32_t find_request(const int64_t* offsets, int32_t n, int64_t b,
                                                DrawShared& sh) {
  if (threadIdx.x == 0) sh.request = INT32_MAX;
  __syncthreads();
  for (int32_t i = threadIdx.x; i < n; i += kDrawThreads)
    if (__ldcg(offsets + i) <= b && b < __ldcg(offsets + i + 1)) atomicMin(&sh.request, i);
  __syncthreads();
  return sh.request == INT32_MAX ? -1 : sh.request;
}

// The lowest index of an element equal to M.
template <typename Row>
__device__ __forceinline__ int32_t first_equal(const Row& r, float M, DrawShared& sh) {
  int32_t best = INT32_MAX;
  for (int32_t u = r.w_lo + r.lane; u < r.w_hi && best == INT32_MAX; u += 32) {
    const uint4 q = r.unit(u);
    if (Row::largest(q) == M) {
#pragma unroll
      for (int e = Row::EPU - 1; e >= 0; --e)
        if (Row::element(q, e) == M) best = u * Row::EPU + e;
    }
  }
  best = __reduce_min_sync(0xFFFFFFFFu, best);
  if (r.lane < r.nrank)
    *peer(&sh.count[r.rank * kDrawWarps + r.warp], r.lane) = (unsigned)best;
  cluster_barrier();
  int32_t all = INT32_MAX;
  for (int q = r.lane; q < r.nrank * kDrawWarps; q += 32) all = min(all, (int32_t)sh.count[q]);
  return __reduce_min_sync(0xFFFFFFFFu, all);
}

// What K is cut by: the first `k` elements; those with less than m before
// them, m somewhere in [m_lo, m_hi].
struct Cut {
  unsigned k;
  u64 m_lo, m_hi;
};

// The CTA's lists as one, in their order, in rank 0's sh.row.list: `n_seg` lists
// with lengths sh.count[], list s at own + (s % per) * stride of rank s / per.
// Returns the number of entries, or -1 where a list or the whole runs over.
__device__ __forceinline__ int gather(DrawShared& sh, int n_seg, int per, int stride) {
  const int tid = threadIdx.x;
  unsigned* off = reinterpret_cast<unsigned*>(sh.wmax);
  unsigned c = tid < n_seg ? sh.count[tid] : 0u;
  const bool bad = c > (unsigned)stride;
  unsigned incl = bad ? 0u : c;
  u64 none = 0ull;
  cta_scan(incl, none, sh);
  if (tid < n_seg) off[tid] = incl - (bad ? 0u : c);
  if (tid == kDrawThreads - 1) sh.all_c = incl;
  if (__syncthreads_or(bad ? 1 : 0) || sh.all_c > (unsigned)kRowList) return -1;
  const int n = (int)sh.all_c;
  for (int g = tid; g < n; g += kDrawThreads) {
    int lo = 0, hi = n_seg;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (off[mid] <= (unsigned)g)
        lo = mid;
      else
        hi = mid;
    }
    sh.row.list[g] = peer(sh.own, lo / per)[(lo % per) * stride + (g - (int)off[lo])];
  }
  __syncthreads();
  return n;
}

// The lists that landed at rank 0, in the order of their warps, in sh.row.list.
// Returns the number of entries, or -1 where one did not fit; *coarse: some
// warp's tail is.
constexpr unsigned kCoarse = 1u << 30;
__device__ __forceinline__ int in_order(DrawShared& sh, int n_seg, bool* coarse) {
  const int tid = threadIdx.x;
  unsigned c = tid < n_seg ? sh.count[tid] : 0u;
  const bool bad = c == 0xFFFFFFFFu;
  const bool rough = !bad && (c & kCoarse);
  c &= kCoarse - 1u;
  unsigned incl = bad ? 0u : c;
  u64 none = 0ull;
  cta_scan(incl, none, sh);
  unsigned* off = reinterpret_cast<unsigned*>(sh.wmax);
  if (tid < n_seg) off[tid] = incl - (bad ? 0u : c);
  if (tid == kDrawThreads - 1) sh.all_c = incl;
  *coarse = __syncthreads_or(rough ? 1 : 0) != 0;
  if (__syncthreads_or(bad ? 1 : 0)) return -1;
  for (int s = tid >> 5; s < n_seg; s += kDrawWarps)
    for (unsigned j = tid & 31; j < (sh.count[s] & (kCoarse - 1u)); j += 32)
      sh.row.list[off[s] + j] = sh.row.landed[sh.landed_at[s] + j];
  __syncthreads();
  return (int)sh.all_c;
}

// Rank 0, on the n entries of sh.row.list, which are in [x_lo, x_hi] and come
// after above_c elements of mass above_m: where K ends, in sh.key, sh.last and
// sh.sum. False: it cannot be told. `complete`: the list holds all elements that
// the floor leaves. Every thread calls it; w[] are the weights of its entries
// (threadIdx.x * per + i).
__device__ __forceinline__ bool settle(DrawShared& sh, int n, int per, const u64 (&w)[3],
                                       unsigned above_c, u64 above_m, const Cut& cut, float x_lo,
                                       float x_hi, bool complete) {
  const int tid = threadIdx.x;
  const float step = (float)(kListBins - 1) / (x_hi - x_lo);
  auto bin_of = [&](float x) {
    return max(0, min(kListBins - 1, (int)((x_hi - x) * step)));
  };
  sh.row.bin.mass[tid] = 0ull;
  sh.row.bin.count[tid] = 0u;
  if (tid == 0) {
    sh.sel[0] = kListBins;
    sh.sel[1] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int j = tid * per + i;
    if (i < per && j < n) {
      const int b = bin_of(__uint_as_float(sh.row.list[j].x));
      atomicAdd(&sh.row.bin.count[b], 1u);
      atomicAdd(&sh.row.bin.mass[b], w[i]);
    }
  }
  __syncthreads();
  const unsigned c = sh.row.bin.count[tid];
  const u64 m = sh.row.bin.mass[tid];
  unsigned ic = c;
  u64 im = m;
  cta_scan(ic, im, sh);
  if (above_c + ic >= cut.k || above_m + im >= cut.m_lo) atomicMin(&sh.sel[0], tid);
  if (tid == kListBins - 1) sh.all_m = above_m + im;
  __syncthreads();
  const int at = sh.sel[0];
  if (at == kListBins) {  // K takes the whole list
    if (tid == 0) {
      sh.key = ordered_bits(x_lo);
      sh.last = INT32_MAX;
      sh.sum = sh.all_m;
    }
    __syncthreads();
    return complete;
  }
  if (tid == at) {
    sh.above_c = above_c + ic - c;
    sh.above_m = above_m + im - m;
    sh.all_c = c;
  }
  __syncthreads();
  const unsigned in_bin = sh.all_c, before_c = sh.above_c;
  const u64 before_m = sh.above_m;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int j = tid * per + i;
    if (i < per && j < n) {
      const uint2 q = sh.row.list[j];
      const float x = __uint_as_float(q.x);
      if (bin_of(x) == at) {
        Ranked e;
        e.w = w[i];
        e.key = ordered_bits(x);
        e.idx = q.y;
        sh.row.last[atomicAdd(&sh.sel[1], 1)] = e;
      }
    }
  }
  __syncthreads();
  // K is a prefix of the bin's elements too: its last one has as many before it
  // as there are others in K.
  unsigned taken = 0u, rank[3];
  u64 mass[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int at_e = tid + i * kDrawThreads;
    bool in = false;
    rank[i] = 0xFFFFFFFFu;
    mass[i] = before_m;
    if (i > 0 && in_bin <= (unsigned)(i * kDrawThreads)) continue;
    if (at_e < (int)in_bin) {
      const Ranked e = sh.row.last[at_e];
      unsigned before = 0u;
#pragma unroll 4
      for (unsigned j = 0; j < in_bin; ++j) {
        const Ranked o = sh.row.last[j];
        if (o.key > e.key || (o.key == e.key && o.idx < e.idx)) {
          ++before;
          mass[i] += o.w;
        }
      }
      in = before_c + before < cut.k && mass[i] < cut.m_lo;
      if (in) rank[i] = before;
    }
    taken += (unsigned)__syncthreads_count(in ? 1 : 0);
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (rank[i] != 0xFFFFFFFFu && rank[i] + 1u == taken) {
      const Ranked e = sh.row.last[tid + i * kDrawThreads];
      sh.key = e.key;
      sh.last = (int32_t)e.idx;
      sh.sum = mass[i] + e.w;
    }
  }
  __syncthreads();
  // cut by the mass: the next element must be out for every m in question
  return before_c + taken >= cut.k || sh.sum >= cut.m_hi;
}

// The sum of 2^(x r - c) over a unit, in binary32; t[] gets its terms.
template <typename Row>
__device__ __forceinline__ float unit_tail(const uint4& q, F2 rh, F2 rl, F2 nc,
                                           F2 (&t)[Row::EPU / 2]) {
#pragma unroll
  for (int e = 0; e < Row::EPU / 2; ++e) {
    const F2 x = f2(Row::element(q, 2 * e), Row::element(q, 2 * e + 1));
    float y0, y1;
    split(fma2(x, rl, fma2(x, rh, nc)), y0, y1);
    t[e] = f2(ex2_approx(y0), ex2_approx(y1));
  }
  F2 s[Row::EPU / 2];
#pragma unroll
  for (int e = 0; e < Row::EPU / 2; ++e) s[e] = t[e];
#pragma unroll
  for (int o = Row::EPU / 4; o > 0; o >>= 1)
#pragma unroll
    for (int e = 0; e < o; ++e) s[e] = add2(s[e], s[e + o]);
  float s0, s1;
  split(s[0], s0, s1);
  return s0 + s1;
}

// A binary32 sum with what its roundings left out.
struct Tail {
  float hi = 0.0f, lo = 0.0f;
  __device__ __forceinline__ void add(float t) {
    const float s = __fadd_rn(hi, t), b = __fsub_rn(s, hi);
    lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(t, b));
    hi = s;
  }
};

// A row that its short list does not settle, by the whole cluster: *set, and the
// draw (not VERIFY). top_k 0 and top_p 1: off.
template <bool VERIFY, typename Row>
__device__ __noinline__ void settle_long(const DrawParams& p, const Row& r, DrawShared& sh,
                                         int64_t b, float M, float T, float floor_x, int32_t top_k,
                                         float top_p, int buf, RowSet* out) {
  constexpr int DT = Row::kDT, ZB = KeyBits<DT>::kZB;
  const int tid = threadIdx.x;
  const WeightRow w = weight_row(M, T, p.drop);
  const uint32_t table = smem_addr(sh.table);
  const bool k_on = top_k >= 1, p_on = top_p < 1.0f;
  const uint32_t floor_key = ordered_bits(floor_x);
  RowSet set = *out;
  Cut cut;
  cut.k = k_on ? (unsigned)top_k : 0xFFFFFFFFu;
  cut.m_lo = cut.m_hi = ULLONG_MAX;
  const u64 p_part = fraction_of(top_p);
  bool settled = false;
  int summed = -1;  // the buffer with the warps' sums of K's weights
  if (!(k_on || p_on)) {
    const u64 own = w.shift ? sum_from<true>(r, w, table, floor_x)
                            : sum_from<false>(r, w, table, floor_x);
    set.sum = cluster_sum(own, r, sh, buf);
    summed = buf;
    buf ^= 1;
    settled = true;
  }

  if (!settled) {
    // Long sets. The histogram's steps run down 32 powers of two for a mass (what
    // lies below counts as nothing: V 2^-32 of the largest weight at most), to
    // the floor for a count.
    const float low = p_on ? fmaxf(floor_x, fmaf(-22.1807098f, T, M)) : floor_x;
    const float step = (float)(kBins - 1) / (M - low);
    for (int j = tid; j < kBins; j += kDrawThreads) sh.hist[j] = 0u;
    __syncthreads();
    // The first four powers of two are weighed exactly: a few heavy elements, whose
    // places in their steps would not average out.
    const float drop = w.rh * w.scale / step;  // powers of two a step
    const int heavy = (int)fminf(4.0f / drop, (float)kBins);
    u64 head = 0ull;
    r.each([&](float x, int32_t) {
      if (x >= floor_x) {
        const int at = max(0, min(kBins - 1, (int)((M - x) * step)));
        atomicAdd(&sh.hist[at], 1u);
        if (at < heavy) head += weight_of(x, w, table);
      }
    });
    head = cluster_sum(head, r, sh, buf);  // (its barrier ends the histograms)
    buf ^= 1;
    // each CTA adds up its share of the steps and hands the sums to all
    const int share = (kBins / 4 + r.nrank - 1) / r.nrank;
    for (int j = tid; j < share; j += kDrawThreads) {
      const int at = r.rank * share + j;
      if (at < kBins / 4) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 4
        for (int q = 0; q < r.nrank; ++q) {
          const uint4 o = reinterpret_cast<const uint4*>(peer(sh.hist, q))[at];
          v.x += o.x;
          v.y += o.y;
          v.z += o.z;
          v.w += o.w;
        }
        for (int q = 0; q < r.nrank; ++q) reinterpret_cast<uint4*>(peer(sh.steps, q))[at] = v;
      }
    }
    cluster_barrier();
    constexpr int kPer = kBins / kDrawThreads;
    unsigned c[kPer];
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(sh.steps)[tid * (kPer / 4) + i];
      c[4 * i] = v.x;
      c[4 * i + 1] = v.y;
      c[4 * i + 2] = v.z;
      c[4 * i + 3] = v.w;
    }
    // Counts, and masses as if every logit were in the middle of its step, in
    // units of 2^-32: an estimate that the exact masses are held against.
    const float top = (w.shift ? 0.0f : fmaf(M, w.rh, -w.c)) + 32.0f - 0.5f * drop;
    auto middle = [&](int bin, unsigned n) {
      return __float2ull_rn((float)n * ex2_approx(top - (float)bin * drop));
    };
    unsigned own_c = 0u;
    u64 own_m = 0ull, own_h = 0ull;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const u64 m = middle(tid * kPer + i, c[i]);
      own_c += c[i];
      own_m += m;
      if (tid * kPer + i < heavy) own_h += m;
    }
    unsigned none_c = 0u;
    u64 mid_head = own_h;
    cta_scan(none_c, mid_head, sh);
    if (tid == kDrawThreads - 1) sh.above_m = mid_head;
    unsigned end_c = own_c;
    u64 end_m = own_m;
    if (tid < 8) sh.sel[tid] = kBins;
    cta_scan(end_c, end_m, sh);
    if (tid == kDrawThreads - 1) sh.all_m = end_m;
    __syncthreads();
    // what the exact head has over its estimate, added past it
    const u64 more = (head >> 12) - sh.above_m;  // (may be below 0)
    const u64 est = __umul64hi(p_part, sh.all_m + more);
    // The estimate errs by 2e-4 of itself in a row of a hundred (1e-5 in the median):
    // a bracket of 2^-11 either way, or where that holds too many of a quarter.
    const u64 wide = p_on ? est >> 11 : 0ull, slim = wide >> 2;
    unsigned cc = end_c - own_c;
    u64 cm = end_m - own_m;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int bin = tid * kPer + i;
      cc += c[i];
      cm += middle(bin, c[i]);
      const u64 upto = bin + 1 >= heavy ? cm + more : cm;
      if (cc >= cut.k) atomicMin(&sh.sel[0], bin);
      if (p_on) {
        if (upto + wide >= est) atomicMin(&sh.sel[1], bin);
        if (upto >= est + wide) atomicMin(&sh.sel[2], bin);
        if (upto + slim >= est) atomicMin(&sh.sel[3], bin);
        if (upto >= est + slim) atomicMin(&sh.sel[4], bin);
      }
    }
    __syncthreads();
    const int kb = sh.sel[0];
    int b0 = 0, b1 = 0;
    unsigned above_c = 0u;
#pragma unroll 1
    for (int s = 1; s < 5; s += 2) {
      b0 = min(sh.sel[s], kb);
      b1 = min(min(sh.sel[s + 1], kb), kBins - 1);
      // the elements before the bracket and up to its end
      cc = end_c - own_c;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int bin = tid * kPer + i;
        if (bin == b0) sh.above_c = cc;
        cc += c[i];
        if (bin == b1) sh.all_c = cc;
      }
      __syncthreads();
      above_c = b0 < kBins ? sh.above_c : 0u;
      const bool enough = sh.all_c - above_c <= (unsigned)kRowList;
      if (enough) break;
      if (s == 1) __syncthreads();  // the second bracket takes their place
    }
    const bool none = b0 >= kBins;  // top_k alone, and more than there are
    if (none || sh.all_c - above_c <= (unsigned)kRowList) {
      // The exact masses, and the elements of the bracket.
      const float f0 = (float)b0, f1 = b1 == kBins - 1 ? INFINITY : (float)(b1 + 1);
      u64 above = 0ull, all = 0ull, own_above = 0ull;
      WeightSum pa, ps;
      auto list = [&](float x, float v, int32_t i) {
        if (x >= floor_x && v >= f0 && v < f1) {
          const unsigned at = atomicAdd(&sh.own_n, 1u);
          if (at < (unsigned)kCtaList) sh.own[at] = make_uint2(__float_as_uint(x), (uint32_t)i);
        }
      };
      auto sweep = [&](auto shift) {
        r.each_pair(
            [&](float x0, float x1, int32_t i) {
              const float v0 = (M - x0) * step, v1 = (M - x1) * step;
              int32_t h[2], l[2];
              weight_bits<decltype(shift)::value>(x0, x1, w, table, h, l);
              ps.add(h, l);
              const bool a0 = v0 < f0 && x0 >= floor_x, a1 = v1 < f0 && x1 >= floor_x;
              h[0] = a0 ? h[0] : kBitsH;
              h[1] = a1 ? h[1] : kBitsH;
              l[0] = a0 ? l[0] : kBitsL;
              l[1] = a1 ? l[1] : kBitsL;
              pa.add(h, l);
              list(x0, v0, i);
              list(x1, v1, i + 1);
            },
            [&](int n) {
              above += pa.take((uint32_t)n);
              all += ps.take((uint32_t)n);
            });
      };
      if (w.shift)
        sweep(std::true_type{});
      else
        sweep(std::false_type{});
      own_above = warp_sum(above);
      const u64 sa = cluster_sum(above, r, sh, buf);
      const u64 ss = cluster_sum(all, r, sh, buf ^ 1);  // its barrier orders the lists too
      if (p_on) {
        cut.m_lo = cut.m_hi = max(ceil_part(p_part, ss), 1ull);
      }
      if (tid == 0) *peer(&sh.count[r.rank], 0) = sh.own_n;
      cluster_barrier();
      if (r.rank == 0) {
        bool ok = false;
        if (none) {
          if (tid == 0) {
            sh.key = floor_key;
            sh.last = INT32_MAX;
            sh.sum = sa;
          }
          ok = true;
        } else if (!(sa >= cut.m_lo)) {
          const int n = gather(sh, r.nrank, 1, kCtaList);
          if (n >= 0) {
            const int per = (n + kDrawThreads - 1) / kDrawThreads;
            u64 we[3] = {0ull, 0ull, 0ull};
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              const int j = tid * per + i;
              if (i < per && j < n)
                we[i] = weight_of(__uint_as_float(sh.row.list[j].x), w, table);
            }
            float hi = -INFINITY, lo = INFINITY;
            for (int j = tid; j < n; j += kDrawThreads) {
              hi = fmaxf(hi, __uint_as_float(sh.row.list[j].x));
              lo = fminf(lo, __uint_as_float(sh.row.list[j].x));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
              hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
              lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
            }
            if (r.lane == 0) {
              sh.scan_f[r.warp] = hi;
              reinterpret_cast<float*>(sh.scan_m)[r.warp] = lo;
            }
            __syncthreads();
            for (int j = 0; j < kDrawWarps; ++j) {
              hi = fmaxf(hi, sh.scan_f[j]);
              lo = fminf(lo, reinterpret_cast<const float*>(sh.scan_m)[j]);
            }
            __syncthreads();
            ok = settle(sh, n, per, we, above_c, sa, cut, lo, hi, false);
          }
        }
        __syncthreads();
        if (tid < r.nrank) {
          *peer(&sh.key, tid) = sh.key;
          *peer(&sh.last, tid) = sh.last;
          *peer(&sh.sum, tid) = sh.sum;
          *peer(&sh.settled, tid) = ok ? 1 : 0;
        }
      }
      cluster_barrier();
      settled = sh.settled != 0;
      if (settled) {
        set.key = sh.key;
        set.last = sh.last;
        set.sum = sh.sum;
        if constexpr (!VERIFY) {
          // The warps' sums of K: what is above the bracket, and their
          // elements of it that are in K.
          if (r.lane == 0) sh.scan_m[r.warp] = own_above;
          __syncthreads();
          const int n = none ? 0 : (int)sh.own_n;
          for (int j = tid; j < n; j += kDrawThreads) {
            const uint2 q = sh.own[j];
            const float x = __uint_as_float(q.x);
            const uint32_t key = ordered_bits(x);
            if (key > set.key || (key == set.key && (int32_t)q.y <= set.last))
              atomicAdd(&sh.scan_m[r.warp_of((int32_t)q.y)], weight_of(x, w, table));
          }
          __syncthreads();
          cluster_sum(r.lane == 0 ? sh.scan_m[r.warp] : 0ull, r, sh, buf);
          summed = buf;
          buf ^= 1;
        }
      }
    }
  }

  if (!settled) {
    // A radix select.
    if (p_on) {
      const u64 own = w.shift ? sum_from<true>(r, w, table, kLowestLogit)
                              : sum_from<false>(r, w, table, kLowestLogit);
      const u64 all = cluster_sum(own, r, sh, buf);
      buf ^= 1;
      cut.m_lo = max(ceil_part(p_part, all), 1ull);
    }
    unsigned k_rem = cut.k;
    u64 m_rem = cut.m_lo;
    const uint32_t low = floor_key >> ZB;
    const int nb = 32 - __clz((ordered_bits(M) >> ZB) - low);
    uint32_t prefix = 0u;
    unsigned ties = 0u;
    u64 above = 0ull;
    int hb = 0;
    bool reached = true;
    cluster_barrier();  // the histograms take the place of what peers may still read
    for (int hi = nb;;) {
      const int lo = hi > 8 ? hi - 8 : 0;
      if (tid < 256) {
        sh.digit.count[hb][tid] = 0u;
        sh.digit.mass[hb][tid] = 0ull;
      }
      __syncthreads();
      r.each([&](float x, int32_t) {
        if (!(x >= floor_x)) return;
        const uint32_t rel = (ordered_bits(x) >> ZB) - low;
        if (hi < 32 && (rel >> hi) != (prefix >> hi)) return;
        const uint32_t d = (rel >> lo) & ((1u << (hi - lo)) - 1u);
        atomicAdd(&sh.digit.count[hb][d], 1u);
        atomicAdd(&sh.digit.mass[hb][d], weight_of(x, w, table));
      });
      cluster_barrier();
      unsigned c = 0u;
      u64 mass = 0ull;
      if (tid < 256) {
        const int dg = 255 - tid;
        for (int q = 0; q < r.nrank; ++q) {
          c += *peer(&sh.digit.count[hb][dg], q);
          mass += *peer(&sh.digit.mass[hb][dg], q);
        }
      }
      const int d = find_digit(c, mass, k_rem, m_rem, sh);
      if (d < 0) {  // on the first level only: K is all that the floor leaves
        set.sum = sh.all_m;
        reached = false;
        break;
      }
      k_rem -= sh.above_c;
      m_rem -= sh.above_m;
      above += sh.above_m;
      prefix |= (uint32_t)d << lo;
      if (tid == 255 - d) sh.sel[1] = (int)c;
      __syncthreads();
      ties = (unsigned)sh.sel[1];
      hb ^= 1;
      if (lo == 0) break;
      hi = lo;
    }
    if (reached) {
      // The entries on K's last key that K takes.
      const uint32_t key = key_of_short<DT>(low + prefix);
      const u64 each = weight_of(logit_of_key(key), w, table);
      u64 take = k_rem;
      if (each > 0ull) {
        const u64 by_mass = m_rem / each + (m_rem % each != 0ull ? 1ull : 0ull);
        if (by_mass < take) take = by_mass;
      }
      if (take < 1ull) take = 1ull;
      set.key = key;
      if (take < ties) {
        auto tie = [&](float x, int32_t) {
          return x >= floor_x && ordered_bits(x) == key ? 1ull : 0ull;
        };
        u64 n = 0ull;
        r.each([&](float x, int32_t i) { n += tie(x, i); });
        cluster_sum(n, r, sh, buf);
        find_index(r, sh, buf, take - 1ull,
                   [&](float x0, float x1, int32_t i, u64(&v)[2]) {
                     v[0] = tie(x0, i);
                     v[1] = tie(x1, i + 1);
                   },
                   [&](int32_t i, float, u64) {
                     for (int q = 0; q < r.nrank; ++q) *peer(&sh.found, q) = i;
                   });
        buf ^= 1;
        cluster_barrier();
        set.last = sh.found;
      } else {
        take = ties;
      }
      set.sum = above + take * each;
    }
  }

  auto kept = [&](float x, int32_t i) {
    if (!(x >= floor_x)) return false;
    const uint32_t key = ordered_bits(x);
    return key > set.key || (key == set.key && i <= set.last);
  };
  if constexpr (!VERIFY) {
    auto pair = [&](float x0, float x1, int32_t i, u64(&v)[2]) {
      weights_of(kept(x0, i) ? x0 : -INFINITY, kept(x1, i + 1) ? x1 : -INFINITY, w, table, v);
    };
    if (summed < 0) {
      u64 own = 0ull;
      r.each_pair(
          [&](float x0, float x1, int32_t i) {
            u64 v[2];
            pair(x0, x1, i, v);
            own += v[0] + v[1];
          },
          [](int) {});
      cluster_sum(own, r, sh, buf);
      summed = buf;
    }
    const u64 target = __umul64hi(fraction_of(__ldcg(p.uniform + b)), set.sum);
    find_index(r, sh, summed, target, pair, [&](int32_t i, float, u64 v) {
      p.out_idx[b] = i;
      if (p.out_logprob) p.out_logprob[b] = log_ratio(v, set.sum, table);
    });
  }
  *out = set;
}

// Row b. VERIFY: its set goes to p.sets[b], with the outcome of its draft's
// test. Otherwise the draw is made and written.
template <bool VERIFY, typename Row>
__device__ __forceinline__ void settle_row(const DrawParams& p, Row& r, DrawShared& sh,
                                           uint16_t* maxima, int64_t b) {
  constexpr int EPU = Row::EPU, DT = Row::kDT;
  const int tid = threadIdx.x;
  r.place(p, b);
  if (tid < 256) sh.near[tid] = sh.near_all[tid] = 0u;
  if (tid == 0) {
    sh.own_n = 0u;
    sh.landed_n = 0u;
  }
  // the settings of the row, or of its request
  int64_t s = b;
  if constexpr (VERIFY) s = find_request(p.offsets, p.n, b, sh);
  const bool owned = s >= 0;  // the same in every CTA of the cluster
  const float T = owned ? __ldcg(p.temperature + s) : 0.0f;
  int32_t top_k = owned && p.top_k ? __ldcg(p.top_k + s) : 0;
  const float top_p = owned && p.top_p ? __ldcg(p.top_p + s) : 1.0f;
  const float min_p = owned && p.min_p ? __ldcg(p.min_p + s) : 0.0f;
  const bool p_on = top_p < 1.0f && top_p > 0.0f;  // NaN: off
  if (top_p <= 0.0f) top_k = 1;
  const bool k_on = top_k >= 1;
  const bool m_on = min_p > 0.0f && T > 0.0f && T < INFINITY;
  if (m_on && tid == kDrawThreads - 1)
    sh.floor_step = min_p < 1.0f ? (double)T * log((double)min_p) : 0.0;

  const bool unfiltered = !(k_on || p_on || m_on);
  // Rows whose mass is asked for sum their weights in the first sweep, in
  // binary32, relative to 2^c0: the largest of the warp's first logits, as a
  // power of two. (The sum is over all; what is listed later comes off it.)
  const bool tails = T > 0.0f && T < 1e30f && p.phase != kLeftOver && (p_on || unfiltered);
  float scale, rh, rl;
  weight_scale(T, scale, rh, rl);
  // the same factor as a pair with a positive low half: -inf stays -inf
  const float th = rh * 0.99999988079071044921875f, tl = (rh - th) + rl;
  float c0 = 0.0f;
  Tail tail;

  if (!owned) return;

  // The largest logit (NaN counts as -inf). A unit's own maximum is kept in
  // sixteen bits, so that the units to list are found without the row: the
  // second look at 304 KB of logits takes 38 KB of shared memory.
  float M = -INFINITY;
  const bool listing = p.phase != kLeftOver && p.maxima;
  auto first = [&](auto with_tail) {
    // two units at a time, and the next two on their way
    constexpr int kBatch = 2;
    F2 t[EPU / 2];
    const F2 rh2 = f2(th), rl2 = f2(tl);
    F2 nc = f2(0.0f);
    const int32_t pad = r.u_lo + (r.w_hi - r.u_lo + 7) / 8 * 8;  // of the last run
    uint4 next[kBatch];
    auto fetch = [&](int32_t u0) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int32_t u = u0 + 32 * i + r.lane;
        next[i] = Row::no_unit();
        if (u < r.w_hi) next[i] = r.unit(u);
      }
    };
    fetch(r.w_lo);
    if constexpr (decltype(with_tail)::value) {
      float m0 = Row::largest(next[0]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m0 = fmaxf(m0, __shfl_xor_sync(0xFFFFFFFFu, m0, o));
      c0 = rintf(m0 * rh);
      if (!(fabsf(c0) <= 512.0f)) c0 = 0.0f;
      nc = f2(-c0);
    }
#pragma unroll 1
    for (int32_t u0 = r.w_lo; u0 < r.w_hi; u0 += 32 * kBatch) {
      uint4 q[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) q[i] = next[i];
      fetch(u0 + 32 * kBatch);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int32_t u = u0 + 32 * i + r.lane;
        const float m = Row::largest(q[i]);
        M = fmaxf(M, m);
        if (listing && u < pad) maxima[u - r.u_lo] = (uint16_t)Row::short_of(fmaxf(m, -INFINITY));
        if constexpr (decltype(with_tail)::value) tail.add(unit_tail<Row>(q[i], rh2, rl2, nc, t));
      }
    }
  };
  if (tails)
    first(std::true_type{});
  else
    first(std::false_type{});
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  if (r.lane < r.nrank) *peer(&sh.wmax[r.rank * kDrawWarps + r.warp], r.lane) = M;
  cluster_barrier();
  for (int q = r.lane; q < r.nrank * kDrawWarps; q += 32) M = fmaxf(M, sh.wmax[q]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));

  RowSet set;
  set.sum = 1ull;
  set.M = M;
  set.key = 0u;
  set.last = -1;
  set.kind = kNothing;
  set.accepted = 0;
  set.request = (int32_t)s;
  int buf = 0;
  if (M == -INFINITY) {
    // no candidate
  } else if (!(T > 0.0f) || M == INFINITY) {
    // Greedy, or +inf takes all the mass.
    set.kind = kOne;
    set.last = first_equal(r, M, sh);
  } else {
    const WeightRow w = weight_row(M, T, p.drop);
    const uint32_t table = smem_addr(sh.table);
    // The lowest logit that K may hold: min_p's, and no element whose weight is
    // zero, which is never drawn.
    float floor_x = w.lowest;
    if (m_on) {
      // the smallest binary32 number from M + T ln(min_p) up
      const double d = sh.floor_step;
      const float dh = (float)d, dl = (float)(d - (double)dh);
      float f = M + dh;
      const float bb = f - M;
      const float rest = ((M - (f - bb)) + (dh - bb)) + dl;
      if (rest > 0.0f && f < M)
        f = __int_as_float(__float_as_int(f) + (f > 0.0f ? 1 : f < 0.0f ? -1 : 0));
      if (rest > 0.0f && f == 0.0f) f = 1.40129846e-45f;
      floor_x = fminf(fmaxf(floor_x, f), M);
    }
    const uint32_t floor_key = ordered_bits(floor_x);
    set.kind = kSet;
    set.key = floor_key;
    set.last = INT32_MAX;
    set.sum = 0ull;
    Cut cut;
    cut.k = k_on ? (unsigned)top_k : 0xFFFFFFFFu;
    cut.m_lo = cut.m_hi = ULLONG_MAX;
    const u64 p_part = fraction_of(top_p);
    bool settled = false, tested = false;

    if (!w.shift && listing && (tails || !(p_on || unfiltered))) {
      // Short sets: 12 powers of two down; for a top_k without a top_p, whose last
      // elements may weigh next to nothing, 24, and 24 nats at low temperatures.
      float x_lo = fmaxf(floor_x, M - (tails ? 8.3177662f * T : fmaxf(16.6355324f * T, 24.0f)));
      if (k_on && !p_on) {
        // Not more than a top_k needs. The units by what their maxima are at least, in
        // 256 steps over the cluster: those down to the step in which the count
        // reaches top_k hold as many elements.
        const float step = 255.0f / (M - x_lo);
        for (int32_t u = r.w_lo + r.lane * 8; u < r.w_hi; u += 256) {
          const uint4 q = lds128(smem_addr(maxima) + (uint32_t)(u - r.u_lo) * 2u);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float v = Row::at_least(word_of(q, e >> 1) >> ((e & 1) * 16) & 0xFFFFu);
            if (v >= x_lo) atomicAdd(&sh.near[max(0, min(255, (int)((M - v) * step)))], 1u);
          }
        }
        __syncthreads();
        if (tid < 256) {
          const unsigned c = sh.near[tid];
          if (c)
            for (int q = 0; q < r.nrank; ++q) atomicAdd(peer(&sh.near_all[tid], q), c);
        }
        cluster_barrier();
        unsigned c = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) c += sh.near_all[r.lane * 8 + i];
        unsigned incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned t = __shfl_up_sync(0xFFFFFFFFu, incl, o);
          if (r.lane >= o) incl += t;
        }
        const unsigned past = __ballot_sync(0xFFFFFFFFu, incl >= cut.k);
        if (past) {
          const int l = __ffs(past) - 1;
          unsigned upto = __shfl_sync(0xFFFFFFFFu, incl - c, l);
          int at = l * 8;
          while (at < l * 8 + 7 && upto + sh.near_all[at] < cut.k) upto += sh.near_all[at++];
          // (a little below the step's end, whatever the roundings)
          if (at < 255) x_lo = fmaxf(x_lo, M - ((float)at + 1.01f) / step);
        }
      }
      // the units to list, in order
      unsigned* todo = reinterpret_cast<unsigned*>(sh.row.list) + r.warp * kWarpList;
      unsigned n_units = 0u;
      for (int32_t u0 = r.w_lo; u0 < r.w_hi; u0 += 256) {
        const int32_t u = u0 + r.lane * 8;
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        bool hit = false;
        if (u < r.w_hi) {
          q = lds128(smem_addr(maxima) + (uint32_t)(u - r.u_lo) * 2u);
          hit = Row::template largest_short<Row::kHalfMaxima ? 2 : 1>(q) >= x_lo;
        }
        if (__ballot_sync(0xFFFFFFFFu, hit) == 0u) continue;
        unsigned in = 0u;
        if (hit) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t s = word_of(q, e >> 1) >> ((e & 1) * 16) & 0xFFFFu;
            in |= Row::of_short(s) >= x_lo ? 1u << e : 0u;
          }
        }
        const unsigned c = __popc(in);
        unsigned incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned t = __shfl_up_sync(0xFFFFFFFFu, incl, o);
          if (r.lane >= o) incl += t;
        }
        unsigned at = n_units + incl - c;
        n_units += __shfl_sync(0xFFFFFFFFu, incl, 31);
        if (n_units > (unsigned)kWarpList) break;
        for (; in; in &= in - 1u) todo[at++] = (unsigned)(u + __ffs(in) - 1);
      }
      __syncwarp();
      // their elements, a unit a lane
      unsigned mine = n_units > (unsigned)kWarpList ? kWarpList + 1u : 0u;
      for (unsigned i0 = 0; i0 < n_units && mine <= (unsigned)kWarpList; i0 += 32) {
        const bool some = i0 + r.lane < n_units;
        const int32_t u = some ? (int32_t)todo[i0 + r.lane] : 0;
        const uint4 q = some ? r.unit(u) : Row::no_unit();
        unsigned c = 0u;
#pragma unroll
        for (int e = 0; e < EPU; ++e) c += Row::element(q, e) >= x_lo ? 1u : 0u;
        if (tails && c) {
          // the unit off the tail, and what is not listed of it on again
          F2 t[EPU / 2];
          const float all = unit_tail<Row>(q, f2(th), f2(tl), f2(-c0), t);
          float left = 0.0f;
#pragma unroll
          for (int e = 0; e < EPU / 2; ++e) {
            float t0, t1;
            split(t[e], t0, t1);
            left += Row::element(q, 2 * e) >= x_lo ? 0.0f : t0;
            left += Row::element(q, 2 * e + 1) >= x_lo ? 0.0f : t1;
          }
          tail.add(-all);
          tail.add(left);
        }
        unsigned incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned t = __shfl_up_sync(0xFFFFFFFFu, incl, o);
          if (r.lane >= o) incl += t;
        }
        unsigned at = mine + incl - c;
        mine += __shfl_sync(0xFFFFFFFFu, incl, 31);
        if (mine <= (unsigned)kWarpList) {
#pragma unroll
          for (int e = 0; e < EPU; ++e) {
            const float x = Row::element(q, e);
            if (x >= x_lo)
              sh.own[r.warp * kWarpList + at++] =
                  make_uint2(__float_as_uint(x), (uint32_t)(u * EPU + e));
          }
        }
      }
      // To rank 0: the list, where it falls, and the tail in units of 2^-44, exact
      // up to the fraction of C. A NaN or an overflow makes the tail one; the list
      // does not count then.
      const float whole = floorf(w.c);
      const float power = c0 - whole + 44.0f;
      bool odd = !(fabsf(tail.hi) + fabsf(tail.lo) < INFINITY) || !(fabsf(c0 - whole) <= 76.0f);
      // y is rounded more coarsely where 2^c0 is far below the largest weight
      const unsigned coarse = c0 < whole - 40.0f ? kCoarse : 0u;
      odd = __any_sync(0xFFFFFFFFu, odd);
      const float to_units = __int_as_float(((int)(odd ? 0.0f : power) + 127) << 23);
      long long sum = 0;
      if (!odd) sum = __float2ll_rn(tail.hi * to_units) + __float2ll_rn(tail.lo * to_units);
      sum = (long long)warp_sum((u64)sum);
      const u64 t = sum > 0 ? __float2ull_rn((float)sum * ex2_approx(whole - w.c)) : 0ull;
      {
        const int at = r.rank * kDrawWarps + r.warp;
        bool fits = !odd && mine <= (unsigned)kWarpList;
        unsigned to = 0u;
        if (r.lane == 0 && fits && mine > 0u) to = atomicAdd(peer(&sh.landed_n, 0), mine);
        to = __shfl_sync(0xFFFFFFFFu, to, 0);
        fits = fits && to + mine <= (unsigned)kLandList;
        __syncwarp();
        if (fits)
          for (unsigned j = r.lane; j < mine; j += 32)
            *peer(&sh.row.landed[to + j], 0) = sh.own[r.warp * kWarpList + j];
        if (r.lane == 0) {
          *peer(&sh.count[at], 0) = fits ? mine | coarse : 0xFFFFFFFFu;
          *peer(&sh.landed_at[at], 0) = to;
          *peer(&sh.sums[buf][at], 0) = t;
        }
      }
      if (p.phase == kShortOnly) {
        // rank 0 goes on alone; the others make room for the next row's
        cluster_arrive();
        if (r.rank != 0) return;
        cluster_wait();
      } else {
        cluster_barrier();
      }
      bool ok = false;
      if (r.rank == 0) {
        bool rough = false;
        const int n = in_order(sh, r.nrank * kDrawWarps, &rough);
        if (n >= 0) {
          const int per = (n + kDrawThreads - 1) / kDrawThreads;
          u64 we[3] = {0ull, 0ull, 0ull}, own = 0ull;
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const int j = tid * per + i;
            if (i < per && j < n) we[i] = weight_of(__uint_as_float(sh.row.list[j].x), w, table);
            own += we[i];
          }
          u64 incl = own;
          unsigned none = 0u;
          cta_scan(none, incl, sh);
          if (tid == kDrawThreads - 1) sh.all_m = incl;
          __syncthreads();
          const u64 listed = sh.all_m;
          if (tails) {
            if (r.warp == 0) {
              u64 rest = 0ull;
              for (int q = r.lane; q < r.nrank * kDrawWarps; q += 32) rest += sh.sums[buf][q];
              rest = warp_sum(rest);
              if (r.lane == 0) {
                // The binary32 tail. In 2^-24 of a term: 23 for y, whose two roundings
                // are of 2^-20 while |y| < 32 (46 where 2^c0 lies more than 40 powers
                // below the largest weight: |y| < 64; terms below either are less than the
                // V units), 4 for ex2, 4 for the sum of a unit, 6 for its scale; then what
                // the rounding of the low parts left of the terms that were listed, and
                // half a unit for each fixed-point weight.
                const float rel = rough ? 64.0f : 40.0f;
                const u64 err = __float2ull_ru((float)rest * (rel * 5.9604645e-8f)) +
                                (listed >> 34) + (u64)p.V;
                sh.tail = rest;
                sh.tail_err = err;
                sh.m_lo = max(ceil_part(p_part, listed + rest - min(rest, err)), 1ull);
                sh.m_hi = ceil_part(p_part, listed + rest + err);
              }
            }
            __syncthreads();
          }
          const u64 rest = tails ? sh.tail : 0ull, err = tails ? sh.tail_err : 0ull;
          if (p_on) {
            cut.m_lo = sh.m_lo;
            cut.m_hi = sh.m_hi;
          }
          const bool complete = x_lo == floor_x;
          if (k_on || p_on) {
            ok = settle(sh, n, per, we, 0u, 0ull, cut, x_lo, M, complete);
          } else if (unfiltered && VERIFY) {
            // The mass is known to err: enough for the draft's test, unless u q S
            // and the draft's weight are that close. (The sum itself, which the draw may
            // need, is formed there: 0 stands for it.)
            if (tid == 0) {
              sh.sel[2] = 1;
              sh.sel[3] = 0;
              const int64_t d = __ldcg(p.draft + b);
              if (b + 1 < __ldcg(p.offsets + s + 1) && b + 1 < p.B && d >= 0 && d < p.V) {
                const float u = fminf(fmaxf(__ldcg(p.uniform + b), 0.0f), 0.999999940395355224609375f);
                const float q = p.probs ? __ldcg(p.probs + b * p.probs_ld + d) : 1.0f;
                const u64 wd = weight_of(logit_at<DT>(r.row, d), w, table);
                const u64 sum = listed + rest;
                const double uq = (double)u * (double)q;
                const bool least = uq * (double)(sum - min(sum, err)) >= (double)wd;
                const bool most = uq * (double)(sum + err) >= (double)wd;
                sh.sel[2] = wd == 0ull || least == most;
                sh.sel[3] = wd > 0ull && !most;
              }
            }
            __syncthreads();
            ok = sh.sel[2] != 0;
            tested = true;
            set.accepted = sh.sel[3];
            if (tid == 0) {
              sh.key = floor_key;
              sh.last = INT32_MAX;
              sh.sum = 0ull;
            }
            __syncthreads();
          } else if (unfiltered) {
            // All elements are K. The warp whose run u falls in is told by the
            // listed weights and the tails; in it the weights are exact, and the
            // element stands when u is further from its ends than the error of
            // what lies before.
            u64* run = sh.sums[buf];
            const int segs = r.nrank * kDrawWarps;
            // each warp's listed weights join its tail
            u64 c = 0ull;
            int last = -1;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              const int j = tid * per + i;
              if (i < per && j < n) {
                const int at =
                    r.segment_of((int32_t)sh.row.list[j].y, p.units_per_row, p.units_per_cta);
                if (at != last && c) {
                  atomicAdd(&run[last], c);
                  c = 0ull;
                }
                last = at;
                c += we[i];
              }
            }
            if (c) atomicAdd(&run[last], c);
            __syncthreads();
            const u64 f = fraction_of(__ldcg(p.uniform + b));
            const u64 sum = listed + rest;
            const u64 t_lo = __umul64hi(f, sum - min(sum, err)), t_hi = __umul64hi(f, sum + err);
            const u64 here = tid < segs ? run[tid] : 0ull;
            u64 upto = here;
            cta_scan(none, upto, sh);
            if (tid == 0) sh.sel[0] = -1;
            __syncthreads();
            if (t_lo >= upto - here && t_lo < upto) {
              sh.sel[0] = tid;
              sh.above_m = upto - here;
            }
            __syncthreads();
            const int at = sh.sel[0];
            const u64 before = sh.above_m;
            bool hit = false;
            if (at >= 0 && err <= (sum >> 24)) {
              const int32_t q0 = at / kDrawWarps * p.units_per_cta;
              const int32_t qn = min(p.units_per_cta, p.units_per_row - q0);
              const int32_t each = Row::run_length(qn);
              const int32_t lo = q0 + min(qn, (at % kDrawWarps) * each);
              const int32_t hi = q0 + min(qn, (at % kDrawWarps + 1) * each);
              // (the error of the run's tail is part of err)
              u64 base = before;
              const F2 th2 = f2(th), tl2 = f2(tl), nc = f2(-w.c);
              constexpr float kUnits = 17592186044416.0f;
              for (int32_t u0 = lo; u0 < hi; u0 += kDrawThreads) {
                const int32_t u = u0 + tid;
                uint4 q = Row::no_unit();
                u64 all = 0ull;
                if (u < hi) {
                  q = r.unit(u);
                  F2 t[EPU / 2];
                  const float tails_of = unit_tail<Row>(q, th2, tl2, nc, t);
                  if (Row::largest(q) >= x_lo) {
#pragma unroll 1
                    for (int e = 0; e < EPU; ++e) all += weight_of(Row::element(q, e), w, table);
                  } else {
                    all = __float2ull_rn(tails_of * kUnits);
                  }
                }
                u64 end = all;
                cta_scan(none, end, sh);
                u64 from = base + end - all;
                if (t_lo >= from && t_lo < from + all) {
#pragma unroll 1
                  for (int e = 0; e < EPU; ++e) {
                    const u64 v = weight_of(Row::element(q, e), w, table);
                    if (from + err <= t_lo && t_hi + err < from + v) {
                      hit = true;
                      p.out_idx[b] = u * EPU + e;
                      if (p.out_logprob) p.out_logprob[b] = log_ratio(v, sum, table);
                    }
                    from += v;
                  }
                }
                if (tid == kDrawThreads - 1) sh.all_m = end;
                __syncthreads();
                base += sh.all_m;
                __syncthreads();
              }
            }
            ok = __syncthreads_or(hit ? 1 : 0) != 0;
          } else {
            if (tid == 0) {
              sh.key = floor_key;
              sh.last = INT32_MAX;
              sh.sum = listed;
            }
            __syncthreads();
            ok = complete;
          }
          if (ok && !VERIFY && !unfiltered) {
            // The draw, in the list's order, which is the indices'.
            const uint32_t key = sh.key;
            const int32_t last = sh.last;
            const u64 sum = sh.sum;
            u64 kept = 0ull;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              const int j = tid * per + i;
              if (i < per && j < n) {
                const uint2 q = sh.row.list[j];
                const uint32_t kj = ordered_bits(__uint_as_float(q.x));
                if (kj < key || (kj == key && (int32_t)q.y > last)) we[i] = 0ull;
              }
              kept += we[i];
            }
            const u64 target = __umul64hi(fraction_of(__ldcg(p.uniform + b)), sum);
            u64 end = kept;
            cta_scan(none, end, sh);
            u64 c = end - kept;
            if (target >= c && target < end) {
#pragma unroll
              for (int i = 0; i < 3; ++i) {
                if (target >= c && target < c + we[i]) {
                  const int j = tid * per + i;
                  p.out_idx[b] = (int64_t)sh.row.list[j].y;
                  if (p.out_logprob)
                    p.out_logprob[b] = log_ratio(we[i], sum, table);
                }
                c += we[i];
              }
            }
          }
        }
        if (p.phase != kShortOnly && tid < r.nrank) *peer(&sh.settled, tid) = ok ? 1 : 0;
      }
      if (p.phase == kShortOnly) {
        settled = ok;
      } else {
        cluster_barrier();
        settled = sh.settled != 0;
      }
      buf ^= 1;
      if (settled) {
        if (VERIFY && r.rank == 0) {
          set.key = sh.key;
          set.last = sh.last;
          set.sum = sh.sum;
        }
      }
    }

    if (p.phase == kShortOnly && !settled) {
      // left to a second launch
      if (r.rank == 0 && tid == 0) {
        if constexpr (VERIFY)
          p.sets[b].kind = kOpen;
        else
          p.out_idx[b] = kOpenIndex;
      }
      return;
    }
    if (!settled) {
      tested = false;
      set.accepted = 0;
      settle_long<VERIFY>(p, r, sh, b, M, T, floor_x, k_on ? top_k : 0, p_on ? top_p : 1.0f, buf,
                          &set);
    }
    if constexpr (VERIFY) {
      if (r.rank == 0 && tid == 0 && !tested) {
        const int64_t d = __ldcg(p.draft + b);
        if (b + 1 < __ldcg(p.offsets + s + 1) && b + 1 < p.B && d >= 0 && d < p.V) {
          const float x = logit_at<DT>(r.row, d);
          const float u = fminf(fmaxf(__ldcg(p.uniform + b), 0.0f), 0.999999940395355224609375f);
          const float q = p.probs ? __ldcg(p.probs + b * p.probs_ld + d) : 1.0f;
          const uint32_t key = ordered_bits(x);
          const bool kept =
              x >= floor_x && (key > set.key || (key == set.key && (int32_t)d <= set.last));
          const u64 wd = kept ? weight_of(x, w, table) : 0ull;
          if (wd > 0ull && !((double)u * (double)q * (double)set.sum >= (double)wd))
            set.accepted = 1;
        }
      }
    }
  }
  if (r.rank == 0 && tid == 0) {
    if constexpr (VERIFY) {
      if (set.kind == kOne && b + 1 < __ldcg(p.offsets + s + 1) && b + 1 < p.B) {
        // the set is one token: its draft passes for every u (and q up to 1)
        const float u = fminf(fmaxf(__ldcg(p.uniform + b), 0.0f), 0.999999940395355224609375f);
        const int64_t d = __ldcg(p.draft + b);
        const bool same = d == (int64_t)set.last;
        const float q = same && p.probs ? __ldcg(p.probs + b * p.probs_ld + d) : 1.0f;
        set.accepted = same && !((double)u * (double)q >= 1.0) ? 1 : 0;
      }
      p.sets[b] = set;
    } else if (set.kind != kSet) {
      p.out_idx[b] = set.kind == kOne ? set.last : -1;
      if (p.out_logprob) p.out_logprob[b] = set.kind == kOne ? 0.0f : -INFINITY;
    }
  }
  // No CTA leaves while another may reach its shared memory. (In a kShortOnly
  // launch none does from here on.)
  if (p.phase != kShortOnly) cluster_barrier();
}

// One cluster a row; a kLeftOver launch has fewer, which take the rows that are
// open in turn.
template <int DT, bool VEC, bool VERIFY>
__global__ void __launch_bounds__(kDrawThreads, 2) filter_set_kernel(
    const __grid_constant__ DrawParams p) {
  extern __shared__ __align__(16) uint16_t maxima[];
  __shared__ DrawShared sh;
  cluster_arrive();
  RowCtx<DT, VEC> r;
  r.rank = (int)cg::this_cluster().block_rank();
  r.nrank = p.cluster;
  r.warp = threadIdx.x >> 5;
  r.lane = threadIdx.x & 31;
  if (threadIdx.x < kExp2Entries) sh.table[threadIdx.x] = exp2_entry(threadIdx.x);
  pdl_wait_then_release();
  cluster_wait();  // every CTA of the cluster runs, before the first write to another
  int64_t b = blockIdx.x / r.nrank;
  if (p.phase != kLeftOver) {
    settle_row<VERIFY>(p, r, sh, maxima, b);
    return;
  }
  // 32 rows' flags at a time; every warp of the cluster sees the same ones (a row's
  // is written behind barriers that come after all have read it)
  const int64_t step = gridDim.x / r.nrank;
  for (; b < p.B; b += 32 * step) {
    const int64_t at = b + r.lane * step;
    bool mine = false;
    if (at < p.B)
      mine = VERIFY ? __ldcg(&p.sets[at].kind) == kOpen : __ldcg(p.out_idx + at) == kOpenIndex;
    for (unsigned open = __ballot_sync(0xFFFFFFFFu, mine); open; open &= open - 1u) {
      __syncthreads();
      settle_row<VERIFY>(p, r, sh, maxima, b + (__ffs(open) - 1) * step);
    }
  }
}

// What of a weight exceeds q S: S as the pair (sh, sl) in units of 2^-44 of its
// own, q clamped to [0, 1] (NaN: 0), the product rounded to 2^-44 the way the
// weights are.
__device__ __forceinline__ u64 left_of(u64 w, float q, float sh, float sl) {
  q = fminf(fmaxf(q, 0.0f), 1.0f);
  const float p = q * sh;
  if (!(p < 1.25f)) return 0ull;  // weights are below that
  const float e = fmaf(q, sl, fmaf(q, sh, -p));
  const float vh = (p + e) + kMagicH;
  const float vl = (__fsub_rn(p, __fsub_rn(vh, kMagicH)) + e) + kMagicL;
  const long long less = ((long long)(__float_as_int(vh) - kBitsH) << 22) +
                         (long long)(__float_as_int(vl) - kBitsL);
  return (long long)w > less ? w - (u64)less : 0ull;
}

// One cluster per request, after filter_set_kernel has written its rows' sets:
// the accepted drafts, then the draw from the first row whose draft did not
// pass (max(p - q, 0), or p without the draft where there are no draft
// probabilities), or from p of the last row when all did.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kDrawThreads, 2) verify_draw_kernel(const DrawParams p) {
  using Row = RowCtx<DT, VEC>;
  __shared__ DrawShared sh;
  const int tid = threadIdx.x;
  cluster_arrive();
  Row r;
  r.rank = (int)cg::this_cluster().block_rank();
  r.nrank = p.cluster;
  r.warp = tid >> 5;
  r.lane = tid & 31;
  const int64_t i = blockIdx.x / r.nrank;
  if (tid < kExp2Entries) sh.table[tid] = exp2_entry(tid);
  if (tid == 0) sh.found = INT32_MAX;
  pdl_wait_then_release();
  __syncthreads();
  cluster_wait();  // every CTA of the cluster runs
  int64_t r0 = __ldcg(p.offsets + i), r1 = __ldcg(p.offsets + i + 1);
  r0 = r0 > 0 ? r0 : 0;
  r1 = r1 < p.B ? r1 : p.B;
  if (r1 <= r0) {  // the same in every CTA of the cluster
    if (r.rank == 0 && tid == 0) p.out_count[i] = 0;
    return;
  }
  const int32_t rows = (int32_t)(r1 - r0);
  for (int32_t j = tid; j < rows; j += kDrawThreads)
    if (j == rows - 1 || __ldcg(&p.sets[r0 + j].accepted) == 0) {
      atomicMin(&sh.found, j);
      break;
    }
  __syncthreads();
  const int64_t stop = r0 + sh.found;
  const RowSet* from = p.sets + stop;
  RowSet set;
  set.sum = __ldcg(&from->sum);
  set.M = __ldcg(&from->M);
  set.key = __ldcg(&from->key);
  set.last = __ldcg(&from->last);
  set.kind = __ldcg(&from->kind);
  if (r.rank == 0) {
    for (int64_t b = r0 + tid; b < r1; b += kDrawThreads)
      if (b != stop) p.out_idx[b] = b < stop ? __ldcg(p.draft + b) : -1;
    if (tid == 0) {
      p.out_count[i] = (int32_t)(stop - r0) + (set.kind != kNothing ? 1 : 0);
      if (set.kind != kSet) p.out_idx[stop] = set.kind == kOne ? (int64_t)set.last : -1;
    }
  }
  if (set.kind != kSet) return;  // the whole cluster

  r.place(p, stop);
  const WeightRow w = weight_row(set.M, __ldcg(p.temperature + i), p.drop);
  const uint32_t table = smem_addr(sh.table);
  bool rest = stop != r1 - 1;
  const int64_t draft = __ldcg(p.draft + stop);
  const float* q = p.probs ? p.probs + stop * p.probs_ld : nullptr;
  const float least = logit_of_key(set.key);  // K's smallest logit
  auto kept = [&](float x, int32_t at) {
    return (x > least || (x == least && at <= set.last)) && !(rest && !q && at == draft);
  };
  int buf = 0;
  if (rest && q && set.sum == 0ull) {  // of a row without filter, not formed yet
    const u64 own = w.shift ? sum_from<true>(r, w, table, kLowestLogit)
                            : sum_from<false>(r, w, table, kLowestLogit);
    set.sum = cluster_sum(own, r, sh, buf);
    buf ^= 1;
  }
  // S 2^-44 as a pair
  const u64 top = set.sum >> 30 << 30;
  const float s_hi = (float)top * 5.684341886080802e-14f;
  const float s_lo =
      (float)(long long)(set.sum - (u64)__float2ull_rn((float)top)) * 5.684341886080802e-14f;
  auto weigh = [&](float x0, float x1, int32_t at, float q0, float q1, u64(&v)[2], auto inlined) {
    const bool k0 = kept(x0, at), k1 = kept(x1, at + 1);
    v[0] = v[1] = 0ull;
    if (!k0 && !k1) return;
    x0 = k0 ? x0 : -INFINITY;
    x1 = k1 ? x1 : -INFINITY;
    if constexpr (decltype(inlined)::value) {
      int32_t h[2], l[2];
      weight_bits<false>(x0, x1, w, table, h, l);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        v[e] = (u64)(((long long)(h[e] - kBitsH) << 22) + (long long)(l[e] - kBitsL));
    } else {
      weights_of(x0, x1, w, table, v);
    }
    if (rest && q) {
      v[0] = left_of(v[0], q0, s_hi, s_lo);
      v[1] = left_of(v[1], q1, s_hi, s_lo);
    }
  };
  auto pair = [&](float x0, float x1, int32_t at, u64(&v)[2]) {
    const bool some = rest && q;
    const float q0 = some && at < p.V ? __ldg(q + at) : 0.0f;
    const float q1 = some && at + 1 < p.V ? __ldg(q + at + 1) : 0.0f;
    weigh(x0, x1, at, q0, q1, v, std::false_type{});
  };
  const bool q_wide = q && ((uintptr_t)q & 15u) == 0;
  u64 all;
  for (;;) {
    u64 own = 0ull;
    auto sweep = [&](auto inlined) {
      uint4 next = r.w_lo + r.lane < r.w_hi ? r.unit(r.w_lo + r.lane) : Row::no_unit();
      for (int32_t u = r.w_lo + r.lane; u < r.w_hi; u += 32) {
        const uint4 c = next;
        if (u + 32 < r.w_hi) next = r.unit(u + 32);
        if (!(Row::largest(c) >= least)) continue;
        const int32_t at = u * Row::EPU;
        float qs[Row::EPU];
#pragma unroll
        for (int e = 0; e < Row::EPU; ++e) qs[e] = 0.0f;
        if (rest && q) {
          if (q_wide && at + Row::EPU <= p.V) {
#pragma unroll
            for (int e = 0; e < Row::EPU; e += 4) {
              const float4 f = __ldg(reinterpret_cast<const float4*>(q + at + e));
              qs[e] = f.x;
              qs[e + 1] = f.y;
              qs[e + 2] = f.z;
              qs[e + 3] = f.w;
            }
          } else {
#pragma unroll
            for (int e = 0; e < Row::EPU; ++e)
              if (at + e < p.V) qs[e] = __ldg(q + at + e);
          }
        }
#pragma unroll
        for (int e = 0; e < Row::EPU; e += 2) {
          u64 v[2];
          weigh(Row::element(c, e), Row::element(c, e + 1), at + e, qs[e], qs[e + 1], v, inlined);
          own += v[0] + v[1];
        }
      }
    };
    if (w.shift)
      sweep(std::false_type{});
    else
      sweep(std::true_type{});
    all = cluster_sum(own, r, sh, buf);
    if (all > 0ull || !rest) break;
    rest = false;  // nothing is left of p - q: the draw is from p
    buf ^= 1;
  }
  const u64 target = __umul64hi(fraction_of(__ldcg(p.uniform_draw + i)), all);
  find_index(r, sh, buf, target, pair, [&](int32_t at, float, u64) { p.out_idx[stop] = at; });
  cluster_barrier();
}

// The kernels of one dtype.
template <int DT>
void* draw_kernel_of(bool vec, bool verify) {
  if (vec)
    return verify ? reinterpret_cast<void*>(&filter_set_kernel<DT, true, true>)
                  : reinterpret_cast<void*>(&filter_set_kernel<DT, true, false>);
  return verify ? reinterpret_cast<void*>(&filter_set_kernel<DT, false, true>)
                : reinterpret_cast<void*>(&filter_set_kernel<DT, false, false>);
}

template <int DT>
void* verify_draw_kernel_of(bool vec) {
  return vec ? reinterpret_cast<void*>(&verify_draw_kernel<DT, true>)
             : reinterpret_cast<void*>(&verify_draw_kernel<DT, false>);
}

}  // namespace
}  // namespace gsample
