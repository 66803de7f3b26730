// Pages of a paged cache: which physical page holds each run of a request
// slot's tokens, kept on the device, where the lengths that a verification of
// drafts leaves are known. Pages are handed out and taken back in the order of
// the requests by prefix sums, so the same calls give the same tables.
//
// All arithmetic is on integers and the work is reading and writing tables and
// maps: an extension is bound by its launches until a batch's maps reach a few
// MB.
#include <climits>
#include <cstdint>

#include "gsample_internal.h"

namespace gsample {
namespace {

constexpr int kPageThreads = 1024;
constexpr int kPageWarps = kPageThreads / 32;
constexpr int kMapThreads = 256;
constexpr int kMapTokens = 1024;  // slot-map entries of a CTA
constexpr int kMapOffsets = 1025;
constexpr int kTableCols = 1024;  // table columns of a CTA at a time

// The list of request i, clipped to [0, total).
struct List {
  int64_t at;
  int64_t count;
};

__device__ __forceinline__ List list_of(const int64_t* offsets, int64_t total, int64_t i) {
  if (!offsets) return List{i, 1};
  const int64_t a = min(max(__ldcg(offsets + i), (int64_t)0), total);
  const int64_t b = min(max(__ldcg(offsets + i + 1), a), total);
  return List{a, b - a};
}

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int32_t page) {
  return (tokens + page - 1) / page;
}

// Inclusive scan of one value per thread over the CTA. Ends with a barrier;
// *total gets the CTA's sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* scratch, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t w = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += t;
    }
    scratch[lane] = w;
  }
  __syncthreads();
  if (warp > 0) v += scratch[warp - 1];
  *total = scratch[kPageWarps - 1];
  __syncthreads();
  return v;
}

// The state row of request i, or -1 where the slot is out of range or named
// more than once. `once` and `more` are bitmaps over the rows in shared memory.
__device__ __forceinline__ void mark_slots(const PageArgs& s, const int32_t* slot, int64_t n,
                                           uint32_t* once, uint32_t* more) {
  if (!slot) return;
  const int64_t words = (s.rows + 31) / 32;
  for (int64_t j = threadIdx.x; j < 2 * words; j += blockDim.x) once[j] = 0u;
  __syncthreads();
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
    const int32_t r = __ldcg(slot + i);
    if (r < 0 || r >= s.rows) continue;
    const uint32_t bit = 1u << (r & 31);
    if (atomicOr(once + (r >> 5), bit) & bit) atomicOr(more + (r >> 5), bit);
  }
  __syncthreads();
}

__device__ __forceinline__ int64_t row_of(const PageArgs& s, const int32_t* slot, int64_t i,
                                          const uint32_t* more) {
  if (!slot) return i;
  const int32_t r = __ldcg(slot + i);
  if (r < 0 || r >= s.rows || (more[r >> 5] >> (r & 31) & 1u)) return -1;
  return r;
}

__device__ __forceinline__ int64_t length_of(const PageArgs& s, int64_t row) {
  const int64_t most = s.ld * s.page_size;
  return min(max((int64_t)__ldcg(s.length + row), (int64_t)0), most);
}

// The last q in [0, m) with first[q] <= j (first[0] <= j, not decreasing).
__device__ __forceinline__ int last_not_above(const int64_t* first, int m, int64_t j) {
  int lo = 0, hi = m;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= j)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The bookkeeping of an extension, one CTA: new pages into the tables, lengths
// and the stack of free pages. Request i of a tile takes the entries
// [first, first + need) below the top of the stack.
__global__ void __launch_bounds__(kPageThreads) pages_extend_kernel(const PageArgs s,
                                                                    const ExtendArgs a) {
  extern __shared__ uint32_t bitmaps[];
  __shared__ int64_t scratch[32];
  __shared__ int64_t first[kPageThreads];
  __shared__ int64_t place[kPageThreads];  // row * ld + pages held
  pdl_wait_then_release();
  uint32_t* more = bitmaps + (s.rows + 31) / 32;
  mark_slots(s, a.slot, a.n, bitmaps, more);
  const int64_t top = min(max((int64_t)__ldcg(s.free_count), (int64_t)0), s.pages);
  int64_t taken = 0;   // pages wanted by the tiles before
  int64_t granted = 0;
  for (int64_t i0 = 0; i0 < a.n; i0 += kPageThreads) {
    const int64_t i = i0 + threadIdx.x;
    int64_t row = -1, need = 0, held = 0, old = 0, count = 0;
    if (i < a.n) {
      row = row_of(s, a.slot, i, more);
      if (row >= 0) {
        old = length_of(s, row);
        count = list_of(a.offsets, a.total, i).count;
        held = pages_of(old, s.page_size);
        if (old + count > s.ld * s.page_size)
          row = -1;
        else
          need = pages_of(old + count, s.page_size) - held;
      }
    }
    int64_t all = 0;
    const int64_t end = taken + block_scan(need, scratch, &all);
    const int64_t begin = end - need;
    if (need > 0 && end > top) {
      row = -1;
      need = 0;
    }
    first[threadIdx.x] = min(begin, top);
    place[threadIdx.x] = row >= 0 ? row * s.ld + held : 0;
    if (i < a.n) {
      a.out_start[i] = row >= 0 ? (int32_t)old : -1;
      if (a.out_length) a.out_length[i] = row >= 0 ? (int32_t)(old + count) : 0;
      if (row >= 0) s.length[row] = (int32_t)(old + count);
    }
    // the pages of the tile's granted requests, which come first
    const int64_t from = min(taken, top);
    int64_t got = 0;
    block_scan(need, scratch, &got);
    for (int64_t j = from + threadIdx.x; j < from + got; j += kPageThreads) {
      const int q = last_not_above(first, kPageThreads, j);
      s.table[place[q] + (j - first[q])] = __ldcg(s.free_list + (top - 1 - j));
    }
    taken += all;
    granted += got;
    __syncthreads();
  }
  if (threadIdx.x == 0) *s.free_count = (int32_t)(top - granted);
}

// The slot map and the batch's block table, from the state after the
// extension: the first `map_ctas` CTAs take kMapTokens entries of the map each,
// the others kTableCols columns of one request's table at a time. What a request
// is gets read once a CTA (a division and four dependent loads an entry took
// 12 us for 256 tables of 2049 columns, this 5), and a token finds its request
// among offsets in shared memory.
__global__ void __launch_bounds__(kMapThreads) pages_map_kernel(const PageArgs s,
                                                                const ExtendArgs a) {
  __shared__ int64_t offsets[kMapOffsets];
  pdl_wait_then_release();
  const uint32_t page = (uint32_t)s.page_size;
  if (blockIdx.x < (unsigned)a.map_ctas) {
    const bool near = a.offsets && a.n + 1 <= kMapOffsets;
    if (near) {
      for (int64_t i = threadIdx.x; i <= a.n; i += kMapThreads) offsets[i] = __ldcg(a.offsets + i);
      __syncthreads();
    }
    auto offset = [&](int64_t i) { return near ? offsets[i] : __ldcg(a.offsets + i); };
    const int64_t t0 = (int64_t)blockIdx.x * kMapTokens;
    const int64_t t1 = min(t0 + kMapTokens, a.total);
    for (int64_t t = t0 + threadIdx.x; t < t1; t += kMapThreads) {
      int64_t i = t, at = t;
      if (a.offsets) {
        if (t < offset(0) || t >= offset(a.n)) continue;
        int64_t lo = 0, hi = a.n;
        while (hi - lo > 1) {
          const int64_t mid = (lo + hi) >> 1;
          if (offset(mid) <= t)
            lo = mid;
          else
            hi = mid;
        }
        i = lo;
        at = min(max(offset(i), (int64_t)0), a.total);
        if (t < at || t >= min(max(offset(i + 1), at), a.total)) continue;
      }
      const int32_t start = __ldcg(a.out_start + i);
      const int64_t row = a.slot ? (int64_t)__ldcg(a.slot + i) : i;
      int64_t where = -1;
      if (start >= 0) {
        const uint32_t position = (uint32_t)start + (uint32_t)(t - at);  // below 2^31
        const uint32_t c = position / page;
        where = (int64_t)__ldcg(s.table + row * s.ld + c) * page + (position - c * page);
      }
      a.out_slot_map[t] = where;
    }
  } else {
    const uint32_t chunks = (uint32_t)((a.table_cols + kTableCols - 1) / kTableCols);
    const int64_t all = a.n * chunks;
    for (int64_t j = blockIdx.x - a.map_ctas; j < all; j += gridDim.x - a.map_ctas) {
      const int64_t i = j / chunks;
      const int64_t c0 = (j - i * chunks) * kTableCols;
      const int64_t c1 = min(c0 + kTableCols, a.table_cols);
      const int32_t start = __ldcg(a.out_start + i);
      const int64_t row = a.slot ? (int64_t)__ldcg(a.slot + i) : i;
      const int64_t count = list_of(a.offsets, a.total, i).count;
      const int64_t held = start >= 0 ? ((uint32_t)start + (uint32_t)count + page - 1) / page : 0;
      const int32_t* from = s.table + (start >= 0 ? row * s.ld : 0);
      int32_t* to = a.out_table + i * a.table_ld;
#pragma unroll 4
      for (int64_t c = c0 + threadIdx.x; c < c1; c += kMapThreads)
        to[c] = c < held ? __ldcg(from + c) : -1;
    }
  }
}

// Shortens slots: the pages past their new lengths go back on the stack, in the
// places that an extension of the same requests takes them from.
__global__ void __launch_bounds__(kPageThreads) pages_trim_kernel(const PageArgs s,
                                                                  const TrimArgs a) {
  extern __shared__ uint32_t bitmaps[];
  __shared__ int64_t scratch[32];
  __shared__ int64_t first[kPageThreads];
  __shared__ int64_t place[kPageThreads];
  pdl_wait_then_release();
  uint32_t* more = bitmaps + (s.rows + 31) / 32;
  mark_slots(s, a.slot, a.n, bitmaps, more);
  const int64_t top = min(max((int64_t)__ldcg(s.free_count), (int64_t)0), s.pages);
  // the new length of request i's row, or -1 where it is left alone
  auto shortened = [&](int64_t i, int64_t* row, int64_t* old) -> int64_t {
    *row = row_of(s, a.slot, i, more);
    if (*row < 0) return -1;
    const int64_t start = a.start ? (int64_t)__ldcg(a.start + i) : 0;
    if (start < 0) return -1;
    const int64_t now = max(start + (a.keep ? (int64_t)__ldcg(a.keep + i) : 0), (int64_t)0);
    *old = length_of(s, *row);
    return now < *old ? now : -1;
  };
  int64_t freed = 0;
  {
    int64_t own = 0;
    for (int64_t i = threadIdx.x; i < a.n; i += kPageThreads) {
      int64_t row, old = 0;
      const int64_t now = shortened(i, &row, &old);
      if (now >= 0) own += pages_of(old, s.page_size) - pages_of(now, s.page_size);
    }
    block_scan(own, scratch, &freed);
  }
  const int64_t new_top = min(top + freed, s.pages);
  int64_t before = 0;
  for (int64_t i0 = 0; i0 < a.n; i0 += kPageThreads) {
    const int64_t i = i0 + threadIdx.x;
    int64_t row = -1, old = 0, now = -1, gone = 0;
    if (i < a.n) {
      now = shortened(i, &row, &old);
      if (now >= 0) gone = pages_of(old, s.page_size) - pages_of(now, s.page_size);
    }
    int64_t all = 0;
    const int64_t end = before + block_scan(gone, scratch, &all);
    first[threadIdx.x] = end - gone;
    place[threadIdx.x] = now >= 0 ? row * s.ld + pages_of(now, s.page_size) : 0;
    if (now >= 0) s.length[row] = (int32_t)now;
    __syncthreads();
    for (int64_t j = before + threadIdx.x; j < before + all; j += kPageThreads) {
      const int q = last_not_above(first, kPageThreads, j);
      int32_t* at = s.table + place[q] + (j - first[q]);
      const int64_t to = new_top - 1 - j;
      if (to >= 0) s.free_list[to] = __ldcg(at);
      *at = -1;
    }
    before += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) *s.free_count = (int32_t)new_top;
}

template <typename K, typename... A>
cudaError_t launch(K kernel, unsigned blocks, int threads, size_t smem, cudaStream_t stream,
                   A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0] = pdl_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

size_t bitmap_bytes(const PageArgs& s, const int32_t* slot) {
  return slot ? (size_t)((s.rows + 31) / 32) * 8 : 0;
}

}  // namespace

cudaError_t launch_pages_extend(const PageArgs& s, ExtendArgs a, int sms, cudaStream_t stream) {
  cudaError_t e = launch(pages_extend_kernel, 1u, kPageThreads, bitmap_bytes(s, a.slot), stream, s, a);
  if (e != cudaSuccess) return e;
  a.map_ctas = (int32_t)((a.total + kMapTokens - 1) / kMapTokens);
  int64_t table_ctas = a.n * ((a.table_cols + kTableCols - 1) / kTableCols);
  if (table_ctas > (int64_t)sms * 8) table_ctas = (int64_t)sms * 8;
  if (a.map_ctas + table_ctas == 0) return cudaSuccess;
  return launch(pages_map_kernel, (unsigned)(a.map_ctas + table_ctas), kMapThreads, 0, stream, s, a);
}

cudaError_t launch_pages_trim(const PageArgs& s, const TrimArgs& a, cudaStream_t stream) {
  return launch(pages_trim_kernel, 1u, kPageThreads, bitmap_bytes(s, a.slot), stream, s, a);
}

}  // namespace gsample

// ---------------------------------------------------------------------------
// Host side: argument checks and status mapping.
// ---------------------------------------------------------------------------
namespace {

using gsample::ExtendArgs;
using gsample::PageArgs;
using gsample::TrimArgs;

constexpr int64_t kMaxRows = int64_t(1) << 16;  // two bitmaps over the rows fit in shared memory

bool misaligned(const void* p, uintptr_t a) { return (uintptr_t)p % a != 0; }

gsample_status check_pages(const gsample_page_state* s, PageArgs* out) {
  if (!s || !s->table || !s->length || !s->free_list || !s->free_count)
    return GSAMPLE_ERR_INVALID_ARG;
  if (misaligned(s->table, 4) || misaligned(s->length, 4) || misaligned(s->free_list, 4) ||
      misaligned(s->free_count, 4))
    return GSAMPLE_ERR_INVALID_ARG;
  if (s->rows < 1 || s->rows > kMaxRows || s->pages < 1 || s->pages > INT32_MAX ||
      s->page_size < 1 || s->ld < 1 || s->ld > INT32_MAX / s->page_size)
    return GSAMPLE_ERR_INVALID_ARG;
  out->table = s->table;
  out->length = s->length;
  out->free_list = s->free_list;
  out->free_count = s->free_count;
  out->rows = s->rows;
  out->ld = s->ld;
  out->pages = s->pages;
  out->page_size = s->page_size;
  return GSAMPLE_OK;
}

gsample_status launched(cudaError_t e) {
  if (e == cudaSuccess) return GSAMPLE_OK;
  cudaGetLastError();
  return GSAMPLE_ERR_CUDA;
}

}  // namespace

extern "C" {

gsample_status gsample_pages_extend(const gsample_page_state* state, const int32_t* slot,
                                    int64_t n, const int64_t* offsets, int64_t total,
                                    int32_t* out_start, int64_t* out_slot_map, int32_t* out_length,
                                    int32_t* out_table, int64_t table_cols, int64_t table_ld,
                                    gsample_stream_t stream) {
  PageArgs s;
  gsample_status st = check_pages(state, &s);
  if (st != GSAMPLE_OK) return st;
  if (n < 0 || n > INT32_MAX || total < 0 || total > INT32_MAX || (!slot && n > s.rows) ||
      (!offsets && total != n))
    return GSAMPLE_ERR_INVALID_ARG;
  if ((n > 0 && !out_start) || (n > 0 && total > 0 && !out_slot_map))
    return GSAMPLE_ERR_INVALID_ARG;
  if (out_table && (table_cols < 0 || table_cols > INT32_MAX || table_ld < table_cols ||
                    table_ld > INT64_MAX / 4 / (n > 0 ? n : 1)))
    return GSAMPLE_ERR_INVALID_ARG;
  if (misaligned(slot, 4) || misaligned(offsets, 8) || misaligned(out_start, 4) ||
      misaligned(out_slot_map, 8) || misaligned(out_length, 4) || misaligned(out_table, 4))
    return GSAMPLE_ERR_INVALID_ARG;
  if (n == 0) return GSAMPLE_OK;
  int sms = 0;
  st = gsample::current_device_sms(&sms);
  if (st != GSAMPLE_OK) return st;
  ExtendArgs a{};
  a.slot = slot;
  a.offsets = offsets;
  a.n = n;
  a.total = total;
  a.out_start = out_start;
  a.out_slot_map = out_slot_map;
  a.out_length = out_length;
  a.out_table = out_table;
  a.table_cols = out_table ? table_cols : 0;
  a.table_ld = table_ld;
  return launched(gsample::launch_pages_extend(s, a, sms, (cudaStream_t)stream));
}

gsample_status gsample_pages_trim(const gsample_page_state* state, const int32_t* slot, int64_t n,
                                  const int32_t* start, const int32_t* keep,
                                  gsample_stream_t stream) {
  PageArgs s;
  gsample_status st = check_pages(state, &s);
  if (st != GSAMPLE_OK) return st;
  if (n < 0 || n > INT32_MAX || (!slot && n > s.rows)) return GSAMPLE_ERR_INVALID_ARG;
  if (misaligned(slot, 4) || misaligned(start, 4) || misaligned(keep, 4))
    return GSAMPLE_ERR_INVALID_ARG;
  if (n == 0) return GSAMPLE_OK;
  int sms = 0;
  st = gsample::current_device_sms(&sms);
  if (st != GSAMPLE_OK) return st;
  TrimArgs a{};
  a.slot = slot;
  a.n = n;
  a.start = start;
  a.keep = keep;
  return launched(gsample::launch_pages_trim(s, a, (cudaStream_t)stream));
}

}  // extern "C"
