// Logit constraints ("Softmax-free GPU sampling: Gumbel-max categorical
// sampling kernel", lablup/mlxcel issue #900, Background: the token bias and
// the repetition / frequency / presence penalties ahead of the sampler; and
// grammar masks): the per-request state and the kernel that writes the
// constrained logits. The draw from them is the samplers' own
// (constrained launches of gsample_sample.cu and gsample_sample_cluster.cu).
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

// One thread per touched word: a word without bits costs its read alone, so
// clearing 64 rows of 151936 that hold some 2000 tokens each takes 5 us, not
// the 12 us that writing their 78 MB would.
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

// The history word and the touched bit of one token, `times` times. Integer
// atomics commute, so the state does not depend on their order.
__device__ __forceinline__ void count_token(const StateArgs& s, int64_t at, uint32_t times,
                                            bool prompt) {
  const uint32_t before =
      prompt ? atomicOr(s.history + at, 0x80000000u) : atomicAdd(s.history + at, times);
  if (before == 0u) atomicOr(s.touched + (at >> 5), 1u << (at & 31));  // ld is a multiple of 32
}

// Where token j's history word is (an index into the whole history), or -1.
__device__ __forceinline__ int64_t token_place(const StateArgs& s, const int32_t* slot, int64_t n,
                                               const int64_t* tokens, const int64_t* offsets,
                                               int64_t j) {
  const int64_t t = __ldcg(tokens + j);  // written by the draw just before, often
  const int64_t i = owner(offsets, n, j);
  if (i < 0 || t < 0 || t >= s.vocab) return -1;
  const int64_t r = state_row(s, slot, i);
  return r < 0 ? -1 : r * s.ld + t;
}

// One thread per token.
__global__ void __launch_bounds__(kConThreads)
    history_append_kernel(const StateArgs s, const int32_t* slot, int64_t n, const int64_t* tokens,
                          int64_t total, const int64_t* offsets, bool prompt) {
  pdl_wait_then_release();
  for (int64_t j = blockIdx.x * (int64_t)kConThreads + threadIdx.x; j < total;
       j += (int64_t)gridDim.x * kConThreads) {
    const int64_t at = token_place(s, slot, n, tokens, offsets, j);
    if (at >= 0) count_token(s, at, 1u, prompt);
  }
}

// Long lists of one request: text repeats its frequent tokens (one in twenty
// is the most frequent one), and atomics on one word of memory run one after
// the other, 2.7 ns each. Here a CTA first counts its kAppendTokens tokens in a
// table in shared memory, where a token takes the first of kAppendProbes places
// that is free or its own (the few that find none go to memory directly), then
// adds each place's count once. Measured for one request of 131072 tokens:
// 11 us, against 21 us one atomic a token; of 32768 5.6 against 6.5, of 16384
// 5.3 against 3.9, so a call of at least kAppendLong tokens a request takes it.
// What is left of the 11 us is latency (table, returning atomics, bits; 13 % of
// the warps, 7 % issue). The lengths are on the device, so the mean decides: one
// list of 131072 among 63 of 300 goes one atomic a token, in 19 us.
constexpr int kAppendTokens = 1024;
constexpr int kAppendSlots = 2048;
constexpr int kAppendProbes = 4;
constexpr int64_t kAppendLong = 32768;

__global__ void __launch_bounds__(kConThreads)
    history_append_long_kernel(const StateArgs s, const int32_t* slot, int64_t n,
                               const int64_t* tokens, int64_t total, const int64_t* offsets,
                               bool prompt) {
  __shared__ unsigned long long key[kAppendSlots];
  __shared__ uint32_t count[kAppendSlots];
  constexpr unsigned long long kEmpty = ~0ull;
  for (int i = threadIdx.x; i < kAppendSlots; i += kConThreads) {
    key[i] = kEmpty;
    count[i] = 0u;
  }
  pdl_wait_then_release();
  __syncthreads();
  for (int64_t j0 = blockIdx.x * (int64_t)kAppendTokens; j0 < total;
       j0 += (int64_t)gridDim.x * kAppendTokens) {
    constexpr int N = kAppendTokens / kConThreads, M = kAppendSlots / kConThreads;
    int64_t at[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int64_t j = j0 + k * kConThreads + threadIdx.x;
      at[k] = j < total ? token_place(s, slot, n, tokens, offsets, j) : -1;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (at[k] < 0) continue;
      const unsigned long long mine = (unsigned long long)at[k];
      uint32_t h = ((uint32_t)at[k] * 2654435761u) >> 21;  // Fibonacci hashing, 11 bits
      int tries = 0;
      for (; tries < kAppendProbes; ++tries, h = (h + 1) % kAppendSlots) {
        const unsigned long long was = atomicCAS(&key[h], kEmpty, mine);
        if (was == kEmpty || was == mine) break;
      }
      if (tries < kAppendProbes)
        atomicAdd(&count[h], 1u);
      else
        count_token(s, at[k], 1u, prompt);
    }
    __syncthreads();
    // All of a thread's additions are on their way before the first is looked at.
    unsigned long long k8[M];
    uint32_t before[M];
#pragma unroll
    for (int k = 0; k < M; ++k) {
      const int i = k * kConThreads + threadIdx.x;
      k8[k] = key[i];
      before[k] = 1u;
      if (k8[k] != kEmpty) {
        before[k] = prompt ? atomicOr(s.history + k8[k], 0x80000000u)
                           : atomicAdd(s.history + k8[k], count[i]);
        key[i] = kEmpty;
        count[i] = 0u;
      }
    }
#pragma unroll
    for (int k = 0; k < M; ++k)
      if (before[k] == 0u) atomicOr(s.touched + (k8[k] >> 5), 1u << (k8[k] & 31));
    __syncthreads();
  }
}

// One warp per request walks its list 32 entries at a time; of the entries of
// a step that name the same token the last one writes, and later steps
// overwrite earlier ones, so the later value stays. Made for lists of up to some
// hundred entries: one of 300 takes 4.4 us, 3000 29 us, 100000 0.9 ms.
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
  constexpr int N = 4;  // steps whose entries are on their way together
  for (int64_t j0 = lo; j0 < hi; j0 += 32 * N) {
    int64_t t[N];
    float v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int64_t j = j0 + k * 32 + lane;
      t[k] = -1;
      v[k] = 0.0f;
      if (j < hi) {
        t[k] = __ldcg(tokens + j);  // both may be what the kernel before wrote
        v[k] = __ldcg(values + j);
        if (t[k] < 0 || t[k] >= s.vocab) t[k] = -1;
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const unsigned same = __match_any_sync(0xFFFFFFFFu, (unsigned long long)t[k]);
      if (t[k] >= 0 && lane == 31 - __clz(same)) {
        s.bias[r * s.ld + t[k]] = v[k];
        atomicOr(s.touched + r * (s.ld / 32) + (t[k] >> 5), 1u << (t[k] & 31));
      }
      __syncwarp();
    }
  }
}

// ---------------------------------------------------------------------------
// Constrained logits
// ---------------------------------------------------------------------------
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

// Two kernels. process_wide_kernel takes rows that all start on 16-byte
// boundaries, process_kernel any others.
//
// process_wide_kernel: a lane takes 32 elements at a time, one word of mask and
// of touched bits, so that what goes by element is a vector instruction or
// nothing: 256-bit loads and stores (a lane's 32 bytes are one sector, so the
// 64-byte stride between lanes costs no traffic), or pairs of 128-bit ones where
// rows start on odd multiples of 16 bytes. Words that the mask leaves
// nothing of are never read. A warp works alone; its words come in groups of
// kWordGroup spread over the row, because the low ids hold most of a request's
// tokens. Touched elements are listed in shared memory and written over their
// places, one a lane, from the logit and the state words fetched for them
// while the words are on their way.
//
// In place, a word is read and written only where the mask takes some but not
// all of it, written only where it takes all, and touched elements are the only
// traffic elsewhere.
//
// Measured at B = 256, V = 151936, bf16 to f32: 42 us without constraints (5.6
// TB/s; the store stream bounds it), 41 with masks, 52 with masks, penalties and
// biases (4.3 TB/s of what that cannot do without; the state words of a touched
// element are two sectors of 32 bytes for its 8). A mask that leaves a few
// tokens, in place: 19 us, 78 MB of stores of which most stay in L2 (22 MB reach
// DRAM within the launch); neither DRAM nor issue (46 %) is full. Eight elements
// a lane took 58 and 23 us, one element 331 and 181. A row's last word, if it is
// cut off, goes element by element through one lane, some 0.35 us each: a single
// f32 row of 50256 takes 8 us, of which process_kernel would need 3.
constexpr int kWideThreads = 128;
constexpr int kWideCtas = 8;     // an SM, 64 registers a thread (80 for binary32 logits)
constexpr int kWideWords = 2;    // words a lane, one after the other
constexpr int kWordGroup = 4;
constexpr int kTouchedCap = 256;  // elements a warp lists at a time

struct Oct {
  uint32_t w[8];
};

// `whole`: p is a multiple of 32; else of 16, and two 128-bit accesses do.
__device__ __forceinline__ Oct ld_oct(const char* p, bool whole) {
  Oct v;
  if (whole) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]),
                   "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
                 : "l"(p)
                 : "memory");
  } else {
    asm volatile(
        "ld.global.v4.b32 {%0, %1, %2, %3}, [%8];\n\t"
        "ld.global.v4.b32 {%4, %5, %6, %7}, [%8 + 16];"
        : "=&r"(v.w[0]), "=&r"(v.w[1]), "=&r"(v.w[2]), "=&r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]),
          "=r"(v.w[6]), "=r"(v.w[7])
        : "l"(p)
        : "memory");
  }
  return v;
}

__device__ __forceinline__ void st_oct(char* p, const Oct& v, bool whole) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.w[0]),
                 "r"(v.w[1]), "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]),
                 "r"(v.w[7])
                 : "memory");
  } else {
    asm volatile(
        "st.global.v4.b32 [%0], {%1, %2, %3, %4};\n\t"
        "st.global.v4.b32 [%0 + 16], {%5, %6, %7, %8};" ::"l"(p),
        "r"(v.w[0]), "r"(v.w[1]), "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]),
        "r"(v.w[7])
        : "memory");
  }
}

// 32 bytes of a row with the elements whose bit in `allowed` is clear set to -inf.
template <int DT>
__device__ __forceinline__ void mask_oct(Oct& v, uint32_t allowed) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (DT == 0) {
      if (!((allowed >> i) & 1u)) v.w[i] = 0xFF800000u;
    } else {
      constexpr uint32_t ninf = (DT == 1 ? 0xFF80u : 0xFC00u) * 0x10001u;
      const uint32_t two = (allowed >> (2 * i)) & 3u;  // the two bits, widened to halves
      const uint32_t keep = ((two | two << 15) & 0x10001u) * 0xFFFFu;
      v.w[i] = (v.w[i] & keep) | (ninf & ~keep);
    }
  }
}

// A listed element on its way: what penalised() needs of it.
struct Gathered {
  int32_t v;
  float l, bias;
  uint32_t h;
};

template <int DT>
__device__ __forceinline__ Gathered gather_element(const ProcessParams& p, int64_t state,
                                                   const char* in, int32_t v) {
  Gathered g;
  g.v = v;
  g.l = logit_at<DT>(in, v);
  g.h = __ldcg(p.con.history + state + v);
  g.bias = p.con.bias ? __ldcg(p.con.bias + state + v) : 0.0f;
  return g;
}

// Writes n listed elements over their places; the next one's gathers are on
// their way while one is written. `g`: the lane's first, gathered already.
template <int DT, int ODT>
__device__ __forceinline__ void write_listed(const ProcessParams& p, int64_t b, int64_t state,
                                             const char* in, char* out, const uint32_t* list,
                                             int n, Gathered g) {
  const int lane = threadIdx.x & 31;
  const RowPenalties pen = row_penalties(p.con, b);
#pragma unroll 1
  for (int i = lane; i < n; i += 32) {
    const Gathered now = g;
    if (i + 32 < n) g = gather_element<DT>(p, state, in, (int32_t)list[i + 32]);
    store_one<ODT>(out, now.v, penalised(now.l, now.h, now.bias, pen));
  }
  __syncwarp();  // before the list is refilled
}

// Where a lane's `mine` elements go in the warp's list, and how many there are
// in all.
struct ListPlace {
  int first, total;
};

__device__ __forceinline__ ListPlace list_place(int mine) {
  if (!__any_sync(0xFFFFFFFFu, mine != 0)) return ListPlace{0, 0};
  const int lane = threadIdx.x & 31;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += up;
  }
  return ListPlace{incl - mine, __shfl_sync(0xFFFFFFFFu, incl, 31)};
}

template <int DT, int ODT, bool INPLACE>
__global__ void __launch_bounds__(kWideThreads, DT == 0 ? 6 : kWideCtas)
    process_wide_kernel(const ProcessParams p) {
  constexpr int ISZ = DT == 0 ? 4 : 2, OSZ = ODT == 0 ? 4 : 2;
  constexpr int NI = ISZ;            // 32-byte pieces of a word's logits
  constexpr int EPO = 32 / ISZ;      // elements a piece
  __shared__ uint32_t lists[kWideThreads / 32][kTouchedCap];
  pdl_wait();  // no release: this kernel writes logits
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t Q = p.warps_per_row;
  const int32_t q = (int32_t)blockIdx.x * (kWideThreads / 32) + warp;
  if (q >= Q) return;
  uint32_t* list = lists[warp];
  const int32_t V = (int32_t)p.V, words = (V + 31) / 32;
  // The lane's k-th word is w0 + k * step: of the warp's 32 / G groups, Q apart.
  constexpr int G = kWordGroup;
  const int32_t w0 = (q + (lane / G) * Q) * G + lane % G, step = 32 * Q;
  for (int64_t b = blockIdx.y; b < p.B; b += gridDim.y) {
    const RowBits r = row_bits(p.con, b);
    const char* in = p.logits + b * p.ld_bytes;
    char* out = p.out + b * p.out_ld_bytes;
#pragma unroll 1
    for (int32_t k = 0; k < p.items_per_lane; ++k) {
      const int32_t w = w0 + k * step;
      const bool whole = w < V / 32;  // the row's last word may be cut off
      uint32_t m = 0u, t = 0u;
      if (w < words) {
        m = r.mask ? __ldcg(reinterpret_cast<const uint32_t*>(r.mask) + w) : 0xFFFFFFFFu;
        if (r.touched) t = __ldcg(reinterpret_cast<const uint32_t*>(r.touched) + w);
      }
      Oct x[NI];
      if (whole && m != 0u && (!INPLACE || m != 0xFFFFFFFFu)) {
#pragma unroll
        for (int i = 0; i < NI; ++i) x[i] = ld_oct(in + (int64_t)w * (32 * ISZ) + i * 32, p.in_by_32);
      }
      // The touched elements, listed, and the first of them on its way, while
      // the word above is.
      const uint32_t todo = whole ? t & m : 0u;
      const ListPlace place = list_place(__popc(todo));
      auto list_round = [&](int base) {  // the elements from the base-th on, as many as it holds
        int at = place.first - base;
        for (uint32_t bits = todo; bits != 0u; bits &= bits - 1u, ++at)
          if (at >= 0 && at < kTouchedCap)
            list[at] = (uint32_t)w * 32u + (uint32_t)__ffs((int)bits) - 1u;
        __syncwarp();
      };
      Gathered g;
      if (place.total != 0) {
        list_round(0);
        if (lane < place.total) g = gather_element<DT>(p, r.state, in, (int32_t)list[lane]);
      }
      if (whole && !(INPLACE && m == 0xFFFFFFFFu)) {
        char* dst = out + (int64_t)w * (32 * OSZ);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (m != 0xFFFFFFFFu) mask_oct<DT>(x[i], m >> (i * EPO));
          if constexpr (DT != 0 && ODT == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              Oct y;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t v = x[i].w[h * 4 + j];
                y.w[2 * j] = __float_as_uint(half_to_f32<DT>(v & 0xFFFFu));
                y.w[2 * j + 1] = __float_as_uint(half_to_f32<DT>(v >> 16));
              }
              st_oct(dst + i * 64 + h * 32, y, p.out_by_32);
            }
          } else {
            st_oct(dst + i * 32, x[i], p.out_by_32);
          }
        }
      }
      if (place.total != 0) {
        __syncwarp();  // orders the words' stores before these elements'
        write_listed<DT, ODT>(p, b, r.state, in, out, list, min(kTouchedCap, place.total), g);
#pragma unroll 1
        for (int base = kTouchedCap; base < place.total; base += kTouchedCap) {
          list_round(base);  // more rounds only where the words are full of touched elements
          const int n = min(kTouchedCap, place.total - base);
          if (lane < n) g = gather_element<DT>(p, r.state, in, (int32_t)list[lane]);
          write_listed<DT, ODT>(p, b, r.state, in, out, list, n, g);
        }
      }
      if (!whole && w < words) {
        const RowConstraints rc = row_constraints(p.con, b);
#pragma unroll 1
        for (int32_t v = w * 32; v < V; ++v) {
          const float l = logit_at<DT>(in, v);
          const float y = constrained_logit(l, v, rc);
          if (!INPLACE || __float_as_uint(l) != __float_as_uint(y)) store_one<ODT>(out, v, y);
        }
      }
    }
  }
}

// process_kernel: row b of the result is cut into units of N elements (N = 8
// for 16-bit logits, 4 for binary32: 16 bytes of the logits) that start on
// 16-byte boundaries of the RESULT, so that every full unit is stored with
// 128-bit stores wherever the two rows start; the first and last unit may be
// partial and go element by element. The logits of a full unit are one 128-bit
// load where they are aligned too; otherwise the two aligned 16-byte pieces
// that hold them, shifted together (both inside the row: units for which they
// are not count as partial).
//
// A warp works alone, as in the wide kernel, on kBatch units a lane at a time:
// groups of kUnitGroup units spread over the row.
constexpr int kProcessCtas = 4;   // an SM: 64 registers a thread (3 and 5: 8 % and 8 % slower)
constexpr int kProcessUnits = 8;  // units a lane at most
constexpr int kBatch = 4;
constexpr int kUnitGroup = 8;

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

template <int DT, int ODT, bool INPLACE>
__global__ void __launch_bounds__(kConThreads, kProcessCtas)
    process_kernel(const ProcessParams p) {
  constexpr int N = DT == 0 ? 4 : 8;
  constexpr int ISZ = DT == 0 ? 4 : 2, OSZ = ODT == 0 ? 4 : 2;
  constexpr uint32_t kFull = (1u << N) - 1u;
  __shared__ uint32_t lists[kConThreads / 32][kTouchedCap];
  pdl_wait();  // no release: this kernel writes logits
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t Q = p.warps_per_row;
  const int32_t q = (int32_t)blockIdx.x * (kConThreads / 32) + warp;
  if (q >= Q) return;
  uint32_t* list = lists[warp];
  const uint64_t pol = evict_first_policy();
  const int32_t V = (int32_t)p.V;
  // The lane's k-th unit is u0 + k * step.
  constexpr int G = kUnitGroup;
  const int32_t u0 = (q + (lane / G) * Q) * G + lane % G, step = 32 * Q;
  for (int64_t b = blockIdx.y; b < p.B; b += gridDim.y) {
    const RowBits r = row_bits(p.con, b);
    const char* in = p.logits + b * p.ld_bytes;
    char* out = p.out + b * p.out_ld_bytes;
    // Elements by which unit 0 starts before the row, and the misalignment of
    // the logits of every unit.
    const int32_t s = (int32_t)((uintptr_t)out & 15u) / OSZ;
    const int a = (int)(((uintptr_t)in - (uintptr_t)(s * ISZ)) & 15u);
    // Full units start in [lo, hi]: all N elements lie in the row, and every
    // byte that is loaded for them (a multiple of ISZ before and after).
    const int32_t lo = a / ISZ, hi = V - (a == 0 ? N : (32 - a) / ISZ);
#pragma unroll 1
    for (int32_t k0 = 0; k0 < p.items_per_lane; k0 += kBatch) {
      int32_t e0[kBatch];
      uint32_t allowed[kBatch], touched[kBatch];
      bool full[kBatch], partial = false;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int32_t u = u0 + (k0 + k) * step;
        const bool in_row = k0 + k < p.items_per_lane && u < p.units_per_row;
        e0[k] = in_row ? u * N - s : V;  // V: neither full nor partial
        full[k] = in_row && e0[k] >= lo && e0[k] <= hi;
        partial |= in_row && !full[k];
        allowed[k] = 0u;
        touched[k] = 0u;
        if (full[k]) {
          allowed[k] = r.mask ? bits_at<N>(r.mask, e0[k]) : kFull;
          if (r.touched) touched[k] = bits_at<N>(r.touched, e0[k]);
        }
      }
      uint4 x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const char* at = in + (int64_t)e0[k] * ISZ;
        if (allowed[k] != 0u && (!INPLACE || allowed[k] != kFull))
          x[k] = a == 0 ? ld_unit(at, pol) : ld_unit_shifted(at, a, pol);
      }
      static_assert(N * kBatch <= 32, "a lane's touched bits fit in one word");
      uint32_t todo = 0u;  // the lane's touched elements, N bits a unit
#pragma unroll
      for (int k = 0; k < kBatch; ++k) todo |= (touched[k] & allowed[k]) << (N * k);
      const ListPlace place = list_place(__popc(todo));
      auto list_round = [&](int base) {
        int at = place.first - base;
        for (uint32_t bits = todo; bits != 0u; bits &= bits - 1u, ++at) {
          const int j = __ffs((int)bits) - 1;
          if (at >= 0 && at < kTouchedCap)
            list[at] = (uint32_t)((u0 + (k0 + j / N) * step) * N - s + j % N);
        }
        __syncwarp();
      };
      Gathered g;
      if (place.total != 0) {
        list_round(0);
        if (lane < place.total) g = gather_element<DT>(p, r.state, in, (int32_t)list[lane]);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (!full[k] || (INPLACE && allowed[k] == kFull)) continue;
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
      if (place.total != 0) {
        __syncwarp();  // orders the units' stores before these elements'
        write_listed<DT, ODT>(p, b, r.state, in, out, list, min(kTouchedCap, place.total), g);
#pragma unroll 1
        for (int base = kTouchedCap; base < place.total; base += kTouchedCap) {
          list_round(base);
          const int n = min(kTouchedCap, place.total - base);
          if (lane < n) g = gather_element<DT>(p, r.state, in, (int32_t)list[lane]);
          write_listed<DT, ODT>(p, b, r.state, in, out, list, n, g);
        }
      }
      if (partial) {  // the units at the row's ends
#pragma unroll 1
        for (int k = 0; k < kBatch; ++k) {
          const int32_t u = u0 + (k0 + k) * step;
          if (k0 + k >= p.items_per_lane || u >= p.units_per_row) break;
          const int32_t e = u * N - s;
          if (e >= lo && e <= hi) continue;
          for (int32_t v = e < 0 ? 0 : e; v < e + N && v < V; ++v) {
            const float l = logit_at<DT>(in, v);
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
  if (total / n >= kAppendLong) {
    const dim3 blocks = blocks_for(total, kAppendTokens, (int64_t)sms * 8);
    return launch(history_append_long_kernel, blocks, kConThreads, stream, s, slot, n, tokens,
                  total, offsets, prompt);
  }
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
  // A warp takes up to kWideWords words, or kProcessUnits units, a lane
  // of a row; fewer while there are not enough warps to fill the device.
  const uintptr_t in_at = (uintptr_t)p.logits | (uintptr_t)p.ld_bytes;
  const uintptr_t out_at = (uintptr_t)p.out | (uintptr_t)p.out_ld_bytes;
  const bool wide = ((in_at | out_at) & 15u) == 0;
  p.in_by_32 = (in_at & 31u) == 0;
  p.out_by_32 = (out_at & 31u) == 0;
  int64_t items, per_warp, slots;
  if (wide) {
    items = ((p.V + 31) / 32 + 31) / 32;
    per_warp = kWideWords;
    slots = (int64_t)sms * kWideCtas * (kWideThreads / 32);
  } else {
    const int64_t n = dtype == 0 ? 4 : 8;
    const int64_t units = (p.V + n - 1) / n + 1;  // the first may start before the row
    items = (units + 31) / 32;
    per_warp = kProcessUnits;
    slots = (int64_t)sms * kProcessCtas * (kConThreads / 32);
    p.units_per_row = (int32_t)units;
  }
  while (per_warp > 1 && p.B * ((items + per_warp - 1) / per_warp) < slots) per_warp /= 2;
  p.warps_per_row = (int32_t)((items + per_warp - 1) / per_warp);
  p.items_per_lane = (int32_t)((items + p.warps_per_row - 1) / p.warps_per_row);
  const int threads = wide ? kWideThreads : kConThreads;
  const int64_t bx = (p.warps_per_row + threads / 32 - 1) / (threads / 32);
  const dim3 grid((unsigned)bx, (unsigned)(p.B < 65535 ? p.B : 65535));
  switch (dtype * 8 + (out_dtype == 0 ? 0 : 4) + (p.inplace ? 2 : 0) + (wide ? 1 : 0)) {
    case 0: return launch(process_kernel<0, 0, false>, grid, threads, stream, p);
    case 1: return launch(process_wide_kernel<0, 0, false>, grid, threads, stream, p);
    case 2: return launch(process_kernel<0, 0, true>, grid, threads, stream, p);
    case 3: return launch(process_wide_kernel<0, 0, true>, grid, threads, stream, p);
    case 8: return launch(process_kernel<1, 0, false>, grid, threads, stream, p);
    case 9: return launch(process_wide_kernel<1, 0, false>, grid, threads, stream, p);
    case 12: return launch(process_kernel<1, 1, false>, grid, threads, stream, p);
    case 13: return launch(process_wide_kernel<1, 1, false>, grid, threads, stream, p);
    case 14: return launch(process_kernel<1, 1, true>, grid, threads, stream, p);
    case 15: return launch(process_wide_kernel<1, 1, true>, grid, threads, stream, p);
    case 16: return launch(process_kernel<2, 0, false>, grid, threads, stream, p);
    case 17: return launch(process_wide_kernel<2, 0, false>, grid, threads, stream, p);
    case 20: return launch(process_kernel<2, 2, false>, grid, threads, stream, p);
    case 21: return launch(process_wide_kernel<2, 2, false>, grid, threads, stream, p);
    case 22: return launch(process_kernel<2, 2, true>, grid, threads, stream, p);
    default: return launch(process_wide_kernel<2, 2, true>, grid, threads, stream, p);
  }
}

}  // namespace gsample
