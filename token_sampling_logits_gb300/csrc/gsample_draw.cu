// The draw from a row's top-k / top-p / min-p set with the caller's random
// number, and the verification of speculative drafts by the same sets.
//
// The set K of a row is a prefix of its candidates (logits that are neither
// NaN nor -inf) in the order (logit descending, index ascending): it ends at
// the first of top_k elements, of the shortest prefix whose softmax mass
// reaches top_p, and of the elements of at least min_p times the largest
// probability. The draw is the inverse CDF over K in index order.
//
// Layout: one thread-block cluster per row, each CTA holding its slice of the
// row in shared memory. Phases, each a pass over the slice and one exchange
// over distributed shared memory:
//   1. the row maximum;
//   2. the row's mass (top_p rows only);
//   3. K's last key by a radix select over order-preserving keys, eight bits a
//      level, with counts and masses (gsample_weights.cuh);
//   4. the last entry on that key that K takes, in index order;
//   5. the draw: the first index whose cumulative weight passes u times K's.
// All sums are integers, so the result does not depend on the order of any
// atomic nor on the split of the row. The only waits are hardware barriers.
#include <cooperative_groups.h>

#include <climits>
#include <cstdint>

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
constexpr size_t kDrawSmemLimit = 100 * 1024;  // two CTAs an SM
constexpr float kLowest = -3.402823466e38f;

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

struct Partial {
  u64 sum;
  float M;
  uint32_t pad;
};

struct DrawShared {
  u64 table[kExp2Entries];
  unsigned hc[2][256];  // digit counts of a level (two buffers)
  u64 hm[2][256];       // digit masses of a level
  u64 wsum[kDrawWarps];
  u64 part[2];          // this CTA's sum, read by the cluster (two buffers)
  float wmax[kDrawWarps];
  float cmax;           // this CTA's largest logit, read by the cluster
  float rowmax;
  u64 before, total;    // the sums before this CTA and of the row
  unsigned sc[8];
  u64 sm[8];
  int sel;
  unsigned above_c, all_c;
  u64 above_m, all_m;
  int32_t found;        // written by the CTA that finds an index
  int32_t request;
};

// One row's work within its cluster: the slice of this CTA and how to read it.
template <int DT, bool VEC, bool RESIDENT>
struct RowCtx {
  using C = HCfg<DT, VEC>;
  static constexpr int EPU = C::kEPU;
  const char* row;
  int32_t V, u_lo, u_hi;
  uint32_t slice;
  int rank, nrank, warp, lane;
  // units of this warp, a contiguous run of the slice, so that warps, CTAs
  // and the unit order within them follow the index order
  int32_t w_lo, w_hi;

  __device__ __forceinline__ uint4 unit(int32_t u) const {
    if constexpr (RESIDENT) {
      return lds128(slice + (uint32_t)(u - u_lo) * 16u);
    } else {
      if constexpr (VEC) {
        if ((u + 1) * EPU <= V) return __ldg(reinterpret_cast<const uint4*>(row) + u);
      }
      return load_unit<DT, VEC>(row, u, V, 0ull);
    }
  }

  static __device__ __forceinline__ float element(const uint4& r, int e) {
    return elt<DT, VEC>(r, e);
  }

  // f(x, i) on every element of this thread's units, in index order.
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
    for (int32_t u = w_lo + lane; u < w_hi; u += 32) {
      const uint4 r = unit(u);
#pragma unroll
      for (int e = 0; e < EPU; ++e) f(elt<DT, VEC>(r, e), u * EPU + e);
    }
  }
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sums v over the cluster: sh.total, and sh.before of the CTAs before this
// one; sh.wsum holds the warps' sums. `buf` alternates between calls: a CTA may
// still read the partial of one call while another writes that of the next.
__device__ __forceinline__ void cluster_sum(u64 v, DrawShared& sh, cg::cluster_group& cluster,
                                            int rank, int nrank, int buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_sum(v);
  if (lane == 0) sh.wsum[warp] = v;
  __syncthreads();
  if (warp == 0) {
    const u64 t = warp_sum(lane < kDrawWarps ? sh.wsum[lane] : 0ull);
    if (lane == 0) sh.part[buf] = t;
  }
  cluster.sync();
  if (warp == 0) {
    const u64 t = lane < nrank ? *cluster.map_shared_rank(&sh.part[buf], lane) : 0ull;
    const u64 all = warp_sum(t);
    const u64 before = warp_sum(lane < rank ? t : 0ull);
    if (lane == 0) {
      sh.total = all;
      sh.before = before;
    }
  }
  __syncthreads();
}

// After cluster_sum of the same weights: the CTA and warp whose run holds the
// element at which the cumulative weight passes `target` (< sh.total) scans it
// and calls done(index, x) in one thread.
template <typename Row, typename W, typename Done>
__device__ __forceinline__ void find_index(const Row& r, const DrawShared& sh, u64 target,
                                           W&& weight, Done&& done) {
  u64 before = sh.before;
  for (int i = 0; i < r.warp; ++i) before += sh.wsum[i];
  if (target < before || target - before >= sh.wsum[r.warp]) return;
  u64 left = target - before;
  for (int32_t u0 = r.w_lo; u0 < r.w_hi; u0 += 32) {
    const int32_t u = u0 + r.lane;
    u64 own = 0ull;
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    if (u < r.w_hi) {
      q = r.unit(u);
#pragma unroll
      for (int e = 0; e < Row::EPU; ++e) own += weight(Row::element(q, e), u * Row::EPU + e);
    }
    u64 incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 t = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (r.lane >= o) incl += t;
    }
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, incl > left);
    if (hit) {
      if (r.lane == __ffs(hit) - 1) {
        u64 c = incl - own;
#pragma unroll 1
        for (int e = 0; e < Row::EPU; ++e) {
          const float x = Row::element(q, e);
          c += weight(x, u * Row::EPU + e);
          if (c > left) {
            done(u * Row::EPU + e, x);
            break;
          }
        }
      }
      return;
    }
    left -= __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
}

// Thread t < 256 holds the totals (c, m) of digit 255 - t. The first digit from
// the top at which the cumulative count reaches k_rem or the cumulative mass
// m_rem (both at least 1), or -1; sh.above_* get the totals above it, sh.all_*
// those of all digits. Called by every thread; ends with a barrier.
__device__ __forceinline__ int find_digit(unsigned c, u64 m, unsigned k_rem, u64 m_rem,
                                          DrawShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) sh.sel = 256;
  unsigned ic = c;
  u64 im = m;
  if (warp < 8) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned tc = __shfl_up_sync(0xFFFFFFFFu, ic, o);
      const u64 tm = __shfl_up_sync(0xFFFFFFFFu, im, o);
      if (lane >= o) {
        ic += tc;
        im += tm;
      }
    }
    if (lane == 31) {
      sh.sc[warp] = ic;
      sh.sm[warp] = im;
    }
  }
  __syncthreads();
  if (warp < 8) {
    for (int i = 0; i < warp; ++i) {
      ic += sh.sc[i];
      im += sh.sm[i];
    }
    if ((ic - c < k_rem && k_rem <= ic) || (im - m < m_rem && m_rem <= im))
      atomicMin(&sh.sel, (int)threadIdx.x);
  }
  __syncthreads();
  const int at = sh.sel;
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

// VERIFY: the row's set goes to p.sets[b], with the outcome of its draft's
// test. Otherwise the draw is made and written.
template <int DT, bool VEC, bool RESIDENT, bool VERIFY>
__global__ void __launch_bounds__(kDrawThreads, 2) filter_set_kernel(const DrawParams p) {
  using Row = RowCtx<DT, VEC, RESIDENT>;
  constexpr int EPU = Row::EPU;
  constexpr int ZB = KeyBits<DT>::kZB;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ DrawShared sh;

  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int nrank = p.cluster;
  const int64_t b = blockIdx.x / nrank;
  for (int j = threadIdx.x; j < kExp2Entries; j += kDrawThreads) sh.table[j] = exp2_entry(j);
  pdl_wait_then_release();

  Row r;
  r.row = p.logits + b * p.ld_bytes;
  r.V = p.V;
  r.u_lo = rank * p.units_per_cta;
  r.u_hi = min(p.units_per_row, r.u_lo + p.units_per_cta);
  r.slice = smem_addr(smem);
  r.rank = rank;
  r.nrank = nrank;
  r.warp = threadIdx.x >> 5;
  r.lane = threadIdx.x & 31;
  {
    const int32_t n = max(0, r.u_hi - r.u_lo), per = (n + kDrawWarps - 1) / kDrawWarps;
    r.w_lo = r.u_lo + min(n, r.warp * per);
    r.w_hi = r.u_lo + min(n, (r.warp + 1) * per);
  }
  if constexpr (RESIDENT) {
    const uint64_t pol = evict_first_policy();
    for (int32_t u = r.w_lo + r.lane; u < r.w_hi; u += 32) {
      const uint32_t dst = r.slice + (uint32_t)(u - r.u_lo) * 16u;
      if (VEC && (u + 1) * EPU <= p.V)
        cp_async16(dst, r.row + (size_t)u * 16, pol);
      else
        sts128(dst, load_unit<DT, VEC>(r.row, u, p.V, pol));
    }
    cp_async_commit();
  }
  // the settings of the row, or of its request
  int64_t s = b;
  if constexpr (VERIFY) s = find_request(p.offsets, p.n, b, sh);
  const bool owned = s >= 0;  // the same in every CTA of the cluster
  const float T = owned ? __ldcg(p.temperature + s) : 0.0f;
  int32_t top_k = owned && p.top_k ? __ldcg(p.top_k + s) : 0;
  float top_p = owned && p.top_p ? __ldcg(p.top_p + s) : 1.0f;
  const float min_p = owned && p.min_p ? __ldcg(p.min_p + s) : 0.0f;
  if constexpr (RESIDENT) cp_async_wait<0>();
  if (!owned) return;

  const bool p_on = top_p < 1.0f && top_p > 0.0f;  // NaN: off
  if (top_p <= 0.0f) top_k = 1;
  const bool k_on = top_k >= 1;

  // 1. The largest logit (NaN counts as -inf).
  float m = -INFINITY;
  r.each([&](float x, int32_t) { m = fmaxf(m, x); });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (r.lane == 0) sh.wmax[r.warp] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kDrawWarps; ++i) m = fmaxf(m, sh.wmax[i]);
    sh.cmax = m;
  }
  cluster.sync();
  if (r.warp == 0) {
    m = r.lane < nrank ? *cluster.map_shared_rank(&sh.cmax, r.lane) : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (r.lane == 0) sh.rowmax = m;
  }
  __syncthreads();
  const float M = sh.rowmax;

  RowSet set;
  set.sum = 0ull;
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
    // Greedy, or +inf takes all the mass: the first element equal to M.
    u64 n = 0ull;
    r.each([&](float x, int32_t) { n += x == M ? 1ull : 0ull; });
    cluster_sum(n, sh, cluster, rank, nrank, buf);
    buf ^= 1;
    find_index(r, sh, 0ull, [&](float x, int32_t) { return x == M ? 1ull : 0ull; },
               [&](int32_t i, float) {
                 for (int q = 0; q < nrank; ++q) *cluster.map_shared_rank(&sh.found, q) = i;
               });
    cluster.sync();
    set.kind = kOne;
    set.last = sh.found;
    set.sum = 1ull;
  } else {
    const WeightRow w = weight_row(M, T, p.fraction_bits);
    const uint32_t table = smem_addr(sh.table);
    // The lowest key that K may hold: min_p's, and no element whose weight is
    // zero (those more than F + 2 < 48 powers of two below M), which is never drawn.
    float floor_x = M - 48.0f * 0.69314718f * T;
    if (min_p > 0.0f) {
      const double d = min_p >= 1.0f ? (double)M : (double)M + (double)T * log((double)min_p);
      if (T < INFINITY) floor_x = fmaxf(floor_x, __double2float_ru(d));
    }
    floor_x = fmaxf(floor_x, kLowest);
    floor_x = fminf(floor_x, M);
    const uint32_t floor_key = ordered_bits(floor_x);
    u64 m_rem = ULLONG_MAX;
    unsigned k_rem = k_on ? (unsigned)top_k : 0xFFFFFFFFu;
    set.kind = kSet;
    set.key = floor_key;
    set.last = INT32_MAX;
    if (p_on) {
      // 2. The row's mass.
      u64 sum = 0ull;
      r.each([&](float x, int32_t) { sum += weight_of(x, w, table); });
      cluster_sum(sum, sh, cluster, rank, nrank, buf);
      buf ^= 1;
      m_rem = ceil_part(fraction_of(top_p), sh.total);
      if (m_rem < 1ull) m_rem = 1ull;
    }
    if (k_on || p_on) {
      // 3. K's last key, relative to the floor.
      const uint32_t low = floor_key >> ZB;
      const int nb = 32 - __clz((ordered_bits(M) >> ZB) - low);
      uint32_t prefix = 0u;
      unsigned ties = 0u;
      u64 above = 0ull;
      int hb = 0;
      bool reached = true;
      for (int hi = nb;;) {
        const int lo = hi > 8 ? hi - 8 : 0;
        if (threadIdx.x < 256) {
          sh.hc[hb][threadIdx.x] = 0u;
          sh.hm[hb][threadIdx.x] = 0ull;
        }
        __syncthreads();
        r.each([&](float x, int32_t) {
          if (!(x >= floor_x)) return;
          const uint32_t rel = (ordered_bits(x) >> ZB) - low;
          if (hi < 32 && (rel >> hi) != (prefix >> hi)) return;
          const uint32_t d = (rel >> lo) & ((1u << (hi - lo)) - 1u);
          atomicAdd(&sh.hc[hb][d], 1u);
          atomicAdd(&sh.hm[hb][d], weight_of(x, w, table));
        });
        cluster.sync();
        unsigned c = 0u;
        u64 mass = 0ull;
        if (threadIdx.x < 256) {
          const int dg = 255 - (int)threadIdx.x;
#pragma unroll 4
          for (int q = 0; q < nrank; ++q) {
            c += *cluster.map_shared_rank(&sh.hc[hb][dg], q);
            mass += *cluster.map_shared_rank(&sh.hm[hb][dg], q);
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
        if ((int)threadIdx.x == 255 - d) sh.sel = (int)c;
        __syncthreads();
        ties = (unsigned)sh.sel;
        hb ^= 1;
        if (lo == 0) break;
        hi = lo;
      }
      if (reached) {
        // 4. The entries on K's last key that K takes.
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
          cluster_sum(n, sh, cluster, rank, nrank, buf);
          buf ^= 1;
          find_index(r, sh, take - 1ull, tie, [&](int32_t i, float) {
            for (int q = 0; q < nrank; ++q) *cluster.map_shared_rank(&sh.found, q) = i;
          });
          cluster.sync();
          set.last = sh.found;
        } else {
          take = ties;
        }
        set.sum = above + take * each;
      }
    }
    auto weight = [&](float x, int32_t i) {
      if (!(x >= floor_x)) return 0ull;
      const uint32_t key = ordered_bits(x);
      if (key < set.key || (key == set.key && i > set.last)) return 0ull;
      return weight_of(x, w, table);
    };
    if (!VERIFY || !(k_on || p_on)) {
      u64 sum = 0ull;
      r.each([&](float x, int32_t i) { sum += weight(x, i); });
      cluster_sum(sum, sh, cluster, rank, nrank, buf);
      set.sum = sh.total;
    }
    if constexpr (!VERIFY) {
      // 5. The draw.
      const u64 target = __umul64hi(fraction_of(__ldcg(p.uniform + b)), set.sum);
      find_index(r, sh, target, weight, [&](int32_t i, float x) {
        p.out_idx[b] = i;
        if (p.out_logprob)
          p.out_logprob[b] = (float)log((double)weight(x, i) / (double)set.sum);
      });
    } else if (rank == 0 && threadIdx.x == 0) {
      const int64_t t = __ldcg(p.draft + b);
      if (b + 1 < __ldcg(p.offsets + s + 1) && b + 1 < p.B && t >= 0 && t < p.V) {
        const float x = logit_at<DT>(r.row, t);
        const float u = fminf(fmaxf(__ldcg(p.uniform + b), 0.0f), 0.999999940395355224609375f);
        const float q = p.probs ? __ldcg(p.probs + b * p.probs_ld + t) : 1.0f;
        const u64 wt = weight(x, (int32_t)t);
        if (wt > 0ull && !((double)u * (double)q * (double)set.sum >= (double)wt)) set.accepted = 1;
      }
    }
  }
  if constexpr (VERIFY) {
    if (rank == 0 && threadIdx.x == 0) {
      if (set.kind == kOne && b + 1 < __ldcg(p.offsets + s + 1) && b + 1 < p.B) {
        // the set is one token: its draft passes for every u
        set.accepted = __ldcg(p.draft + b) == (int64_t)set.last ? 1 : 0;
      }
      p.sets[b] = set;
    }
  } else {
    if (set.kind != kSet && rank == 0 && threadIdx.x == 0) {
      p.out_idx[b] = set.kind == kOne ? set.last : -1;
      if (p.out_logprob) p.out_logprob[b] = set.kind == kOne ? 0.0f : -INFINITY;
    }
  }
  cluster.sync();  // no CTA leaves while another may read its shared memory
}

// q s rounded to an integer, q clamped to [0, 1] (NaN: 0).
__device__ __forceinline__ u64 times_probability(u64 s, float q) {
  const u64 f = __float2ull_rn(fminf(fmaxf(q, 0.0f), 1.0f) * 9223372036854775808.0f);
  const u64 hi = __umul64hi(f, s), lo = f * s;
  return (hi << 1) + (lo >> 63) + ((lo >> 62) & 1ull);
}

// One cluster per request, after filter_set_kernel has written its rows' sets:
// the accepted drafts, then the draw from the first row whose draft did not
// pass (max(p - q, 0), or p without the draft where there are no draft
// probabilities), or from p of the last row when all did.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kDrawThreads, 2) verify_draw_kernel(const DrawParams p) {
  using Row = RowCtx<DT, VEC, false>;
  __shared__ DrawShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int nrank = p.cluster;
  const int64_t i = blockIdx.x / nrank;
  for (int j = threadIdx.x; j < kExp2Entries; j += kDrawThreads) sh.table[j] = exp2_entry(j);
  if (threadIdx.x == 0) sh.found = INT32_MAX;
  pdl_wait_then_release();
  __syncthreads();
  int64_t r0 = __ldcg(p.offsets + i), r1 = __ldcg(p.offsets + i + 1);
  r0 = r0 > 0 ? r0 : 0;
  r1 = r1 < p.B ? r1 : p.B;
  if (r1 <= r0) {  // the same in every CTA of the cluster
    if (rank == 0 && threadIdx.x == 0) p.out_count[i] = 0;
    return;
  }
  const int32_t rows = (int32_t)(r1 - r0);
  for (int32_t j = threadIdx.x; j < rows; j += kDrawThreads)
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
  if (rank == 0) {
    for (int64_t b = r0 + threadIdx.x; b < r1; b += kDrawThreads)
      if (b != stop) p.out_idx[b] = b < stop ? __ldcg(p.draft + b) : -1;
    if (threadIdx.x == 0) {
      p.out_count[i] = (int32_t)(stop - r0) + (set.kind != kNothing ? 1 : 0);
      if (set.kind != kSet) p.out_idx[stop] = set.kind == kOne ? (int64_t)set.last : -1;
    }
  }
  if (set.kind != kSet) return;  // the whole cluster

  Row r;
  r.row = p.logits + stop * p.ld_bytes;
  r.V = p.V;
  r.u_lo = rank * p.units_per_cta;
  r.u_hi = min(p.units_per_row, r.u_lo + p.units_per_cta);
  r.slice = 0u;
  r.rank = rank;
  r.nrank = nrank;
  r.warp = threadIdx.x >> 5;
  r.lane = threadIdx.x & 31;
  {
    const int32_t n = max(0, r.u_hi - r.u_lo), per = (n + kDrawWarps - 1) / kDrawWarps;
    r.w_lo = r.u_lo + min(n, r.warp * per);
    r.w_hi = r.u_lo + min(n, (r.warp + 1) * per);
  }
  const WeightRow w = weight_row(set.M, __ldcg(p.temperature + i), p.fraction_bits);
  const uint32_t table = smem_addr(sh.table);
  bool rest = stop != r1 - 1;
  const int64_t draft = __ldcg(p.draft + stop);
  const float* q = p.probs ? p.probs + stop * p.probs_ld : nullptr;
  auto weight = [&](float x, int32_t at) {
    if (!(x > -INFINITY)) return 0ull;
    const uint32_t key = ordered_bits(x);
    if (key < set.key || (key == set.key && at > set.last)) return 0ull;
    const u64 full = weight_of(x, w, table);
    if (!rest) return full;
    if (!q) return at == draft ? 0ull : full;
    const u64 less = times_probability(set.sum, __ldg(q + at));
    return full > less ? full - less : 0ull;
  };
  int buf = 0;
  for (;;) {
    u64 sum = 0ull;
    r.each([&](float x, int32_t at) { sum += weight(x, at); });
    cluster_sum(sum, sh, cluster, rank, nrank, buf);
    buf ^= 1;
    if (sh.total > 0ull || !rest) break;
    rest = false;  // nothing is left of p - q: the draw is from p
    __syncthreads();
  }
  const u64 target = __umul64hi(fraction_of(__ldcg(p.uniform_draw + i)), sh.total);
  find_index(r, sh, target, weight, [&](int32_t at, float) { p.out_idx[stop] = at; });
  cluster.sync();
}

__global__ void __launch_bounds__(256) debug_weights_kernel(const float* x, int64_t n, float M,
                                                            float T, u64* out) {
  __shared__ u64 tab[kExp2Entries];
  for (int j = threadIdx.x; j < kExp2Entries; j += 256) tab[j] = exp2_entry(j);
  __syncthreads();
  const WeightRow w = weight_row(M, T, 44);
  for (int64_t j = blockIdx.x * (int64_t)256 + threadIdx.x; j < n; j += (int64_t)gridDim.x * 256)
    out[j] = weight_of(x[j], w, smem_addr(tab));
}

template <int DT, bool VEC, bool RES, bool VERIFY>
void* fs() {
  return reinterpret_cast<void*>(&filter_set_kernel<DT, VEC, RES, VERIFY>);
}

template <bool VERIFY>
void* select_set(int dtype, bool vec, bool resident) {
  switch (dtype * 4 + (vec ? 2 : 0) + (resident ? 1 : 0)) {
    case 0: return fs<0, false, false, VERIFY>();
    case 1: return fs<0, false, true, VERIFY>();
    case 2: return fs<0, true, false, VERIFY>();
    case 3: return fs<0, true, true, VERIFY>();
    case 4: return fs<1, false, false, VERIFY>();
    case 5: return fs<1, false, true, VERIFY>();
    case 6: return fs<1, true, false, VERIFY>();
    case 7: return fs<1, true, true, VERIFY>();
    case 8: return fs<2, false, false, VERIFY>();
    case 9: return fs<2, false, true, VERIFY>();
    case 10: return fs<2, true, false, VERIFY>();
    default: return fs<2, true, true, VERIFY>();
  }
}

void* select_verify_draw(int dtype, bool vec) {
  switch (dtype * 2 + (vec ? 1 : 0)) {
    case 0: return reinterpret_cast<void*>(&verify_draw_kernel<0, false>);
    case 1: return reinterpret_cast<void*>(&verify_draw_kernel<0, true>);
    case 2: return reinterpret_cast<void*>(&verify_draw_kernel<1, false>);
    case 3: return reinterpret_cast<void*>(&verify_draw_kernel<1, true>);
    case 4: return reinterpret_cast<void*>(&verify_draw_kernel<2, false>);
    default: return reinterpret_cast<void*>(&verify_draw_kernel<2, true>);
  }
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

void* draw_kernel(int dtype, bool vec, bool resident, int* threads) {
  *threads = kDrawThreads;
  return select_set<false>(dtype, vec, resident);
}

void* verify_kernel(int dtype, bool vec, bool resident, int* threads) {
  *threads = kDrawThreads;
  return select_set<true>(dtype, vec, resident);
}

void* verify_draw_kernel_fn(int dtype, bool vec, bool, int* threads) {
  *threads = kDrawThreads;
  return select_verify_draw(dtype, vec);
}

size_t draw_smem_limit() { return kDrawSmemLimit; }

// One-time per-device setup of the kernels of (dtype, vec): clusters of up to
// 16 CTAs and the full shared-memory slice, then the largest cluster that the
// device co-schedules.
int draw_max_cluster(int dtype, bool vec) {
  int size = kDrawMaxCluster;
  for (int v = 0; v < 5; ++v) {
    const bool res = v & 1;
    void* fn = v == 4 ? select_verify_draw(dtype, vec)
                      : v < 2 ? select_set<false>(dtype, vec, res) : select_set<true>(dtype, vec, res);
    const int smem = v < 4 && res ? (int)kDrawSmemLimit : 0;
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

cudaError_t launch_draw(const DrawParams& p, int dtype, bool vec, cudaStream_t stream) {
  const size_t need = (size_t)p.units_per_cta * 16;
  const bool resident = need <= kDrawSmemLimit;
  void* fn = p.sets ? select_set<true>(dtype, vec, resident) : select_set<false>(dtype, vec, resident);
  return launch_rows(fn, p, p.B, resident ? need : 0, stream);
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
