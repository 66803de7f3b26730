// Host side of the draw from given random numbers and of the verification of
// drafts (include/gsample.h, "Draws from given random numbers"): argument
// checks, launch planning and status mapping. Nothing here touches device data
// or synchronises.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "gsample.h"
#include "gsample_debug.h"
#include "gsample_internal.h"
#include "gsample_weights.cuh"

namespace {

using gsample::DrawParams;

constexpr int kMaxDevices = 64;
constexpr int64_t kUnitsPerCta = 512;  // a CTA of a small batch gets at least this many

int64_t elt_bytes(gsample_dtype dt) { return dt == GSAMPLE_F32 ? 4 : 2; }

bool misaligned(const void* p, uintptr_t a) { return (uintptr_t)p % a != 0; }

gsample_status launched(cudaError_t e) {
  if (e == cudaSuccess) return GSAMPLE_OK;
  cudaGetLastError();
  return GSAMPLE_ERR_CUDA;
}

// The largest cluster of the kernels of (dtype, vec) on the current device.
gsample_status max_cluster(int dtype, bool vec, int* out) {
  static std::mutex mu;
  static int known[kMaxDevices][6];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return GSAMPLE_ERR_CUDA;
  }
  std::lock_guard<std::mutex> lock(mu);
  int& c = known[dev][dtype * 2 + (vec ? 1 : 0)];
  if (c == 0) c = gsample::draw_max_cluster(dtype, vec);
  if (c <= 0) {
    c = 0;
    cudaGetLastError();
    return GSAMPLE_ERR_CUDA;
  }
  *out = c;
  return GSAMPLE_OK;
}

void fill_rows(const void* logits, gsample_dtype dtype, int64_t B, int64_t V, int64_t ld,
               bool vec, DrawParams* p) {
  std::memset(p, 0, sizeof *p);
  p->logits = static_cast<const char*>(logits);
  p->ld_bytes = ld * elt_bytes(dtype);
  p->B = B;
  p->V = (int32_t)V;
  const int epu = gsample::units_elems((int)dtype, vec);
  p->units_per_row = (int32_t)((V + epu - 1) / epu);
  // A row's V weights of little more than 2^44 units at most stay below 2^63.
  int lg = 0;
  while ((int64_t(1) << lg) < V) ++lg;
  p->drop = lg <= 18 ? 0 : lg - 18;
}

void use_cluster(int cluster, DrawParams* p) {
  p->cluster = cluster;
  p->units_per_cta = (p->units_per_row + cluster - 1) / cluster;
}

// The largest cluster size (at most `most`, with at least kUnitsPerCta units a
// CTA) at which `rows` clusters run at once, else 1.
int fitting_cluster(void* fn, bool maxima, int64_t rows, int most, const DrawParams& p) {
  const int64_t nu = p.units_per_row;
  int64_t top = (nu + kUnitsPerCta - 1) / kUnitsPerCta;
  if (top > most) top = most;
  for (int c = (int)top; c > 1; --c) {
    const size_t smem = maxima ? gsample::draw_smem((int32_t)((nu + c - 1) / c)) : 0;
    if (smem > gsample::draw_smem_limit()) break;
    if (rows <= gsample::clusters_at_once(fn, gsample::draw_threads(), c, smem)) return c;
  }
  return 1;
}

// The rows' sets (verification) or draws. With clusters of kOneLaunch CTAs or
// more for all rows at once they take one launch. Otherwise one launch settles
// the short sets, and a second one, with the largest clusters and as many as run
// at once, what is left: a CTA or two would take long for a long row. Measured at
// V = 151936 bf16: 256 rows with one long one 92 us so, 195 with the long row on
// one CTA (62 us without one; the second launch finds nothing in 4 us); 64 long
// rows 91 us in one launch with four CTAs a row, 290 in two. Leaving the last 16
// of 320 rows, which the first launch takes a second wave for, to the second as
// well made 95 us 114.
constexpr int kOneLaunch = 4;
cudaError_t launch_sets(int dtype, bool vec, int64_t rows, int most, DrawParams* p,
                        cudaStream_t stream) {
  void* fn = gsample::draw_kernel(dtype, vec, p->sets != nullptr);
  const size_t limit = gsample::draw_smem_limit();
  int c = fitting_cluster(fn, true, rows, most, *p);
  while (c < most && gsample::draw_smem((p->units_per_row + c - 1) / c) > limit) ++c;
  use_cluster(c, p);
  p->maxima = gsample::draw_smem(p->units_per_cta) <= limit;
  if (c >= kOneLaunch || !p->maxima) return gsample::launch_draw(*p, dtype, vec, rows, stream);
  p->phase = gsample::kShortOnly;
  const cudaError_t e = gsample::launch_draw(*p, dtype, vec, rows, stream);
  if (e != cudaSuccess) return e;
  DrawParams q = *p;
  q.phase = gsample::kLeftOver;
  q.maxima = false;
  use_cluster(fitting_cluster(fn, false, 1, most, q), &q);
  const int64_t n = gsample::clusters_at_once(fn, gsample::draw_threads(), q.cluster, 0);
  return gsample::launch_draw(q, dtype, vec, n < 1 ? 1 : n < rows ? n : rows, stream);
}

}  // namespace

extern "C" {

gsample_status gsample_filtered_categorical(const void* logits, gsample_dtype dtype, int64_t B,
                                            int64_t V, int64_t ld, const float* temperature,
                                            const float* uniform, const int32_t* top_k,
                                            const float* top_p, const float* min_p,
                                            int64_t* out_idx, float* out_logprob,
                                            gsample_stream_t stream) {
  gsample_status st = gsample::check_logits(logits, dtype, B, V, ld);
  if (st != GSAMPLE_OK) return st;
  if (B > 0 && (!temperature || !uniform || !out_idx)) return GSAMPLE_ERR_INVALID_ARG;
  if (misaligned(temperature, 4) || misaligned(uniform, 4) || misaligned(top_k, 4) ||
      misaligned(top_p, 4) || misaligned(min_p, 4) || misaligned(out_idx, 8) ||
      misaligned(out_logprob, 4) || B > INT32_MAX / 16)
    return GSAMPLE_ERR_INVALID_ARG;
  if (B == 0) return GSAMPLE_OK;
  int sms = 0, most = 0;
  st = gsample::current_device_sms(&sms);
  if (st != GSAMPLE_OK) return st;
  const bool vec = gsample::wide_rows(logits, dtype, ld);
  st = max_cluster((int)dtype, vec, &most);
  if (st != GSAMPLE_OK) return st;
  DrawParams p;
  fill_rows(logits, dtype, B, V, ld, vec, &p);
  p.temperature = temperature;
  p.uniform = uniform;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.out_idx = out_idx;
  p.out_logprob = out_logprob;
  try {
    return launched(launch_sets((int)dtype, vec, B, most, &p, (cudaStream_t)stream));
  } catch (...) {
    return GSAMPLE_ERR_CUDA;
  }
}

size_t gsample_verify_workspace_bytes(int64_t R) {
  return R > 0 ? (size_t)R * sizeof(gsample::RowSet) : 0;
}

gsample_status gsample_verify_drafts(const void* logits, gsample_dtype dtype, int64_t R, int64_t V,
                                     int64_t ld, int64_t n, const int64_t* offsets,
                                     const int64_t* draft, const float* draft_probs,
                                     int64_t draft_probs_ld, const float* temperature,
                                     const int32_t* top_k, const float* top_p, const float* min_p,
                                     const float* uniform, const float* uniform_draw,
                                     int64_t* out_tokens, int32_t* out_count, void* workspace,
                                     gsample_stream_t stream) {
  gsample_status st = gsample::check_logits(logits, dtype, R, V, ld);
  if (st != GSAMPLE_OK) return st;
  if (n < 0 || n > INT32_MAX / 16 || R > INT32_MAX / 16) return GSAMPLE_ERR_INVALID_ARG;
  if (n > 0 && (!offsets || !temperature || !uniform_draw || !out_count))
    return GSAMPLE_ERR_INVALID_ARG;
  if (R > 0 && n > 0 && (!draft || !uniform || !out_tokens)) return GSAMPLE_ERR_INVALID_ARG;
  if (draft_probs && (draft_probs_ld < V || draft_probs_ld > INT64_MAX / 4 / (R > 0 ? R : 1)))
    return GSAMPLE_ERR_INVALID_ARG;
  if (misaligned(offsets, 8) || misaligned(draft, 8) || misaligned(draft_probs, 4) ||
      misaligned(temperature, 4) || misaligned(top_k, 4) || misaligned(top_p, 4) ||
      misaligned(min_p, 4) || misaligned(uniform, 4) || misaligned(uniform_draw, 4) ||
      misaligned(out_tokens, 8) || misaligned(out_count, 4))
    return GSAMPLE_ERR_INVALID_ARG;
  if (R > 0 && n > 0 && (!workspace || misaligned(workspace, 16))) return GSAMPLE_ERR_WORKSPACE;
  if (n == 0) return GSAMPLE_OK;
  int sms = 0, most = 0;
  st = gsample::current_device_sms(&sms);
  if (st != GSAMPLE_OK) return st;
  const bool vec = R > 0 && gsample::wide_rows(logits, dtype, ld);
  st = max_cluster((int)dtype, vec, &most);
  if (st != GSAMPLE_OK) return st;
  DrawParams p;
  fill_rows(logits, dtype, R, V, ld, vec, &p);
  p.n = (int32_t)n;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.uniform = uniform;
  p.uniform_draw = uniform_draw;
  p.offsets = offsets;
  p.draft = draft;
  p.probs = draft_probs;
  p.probs_ld = draft_probs_ld;
  p.out_idx = out_tokens;
  p.out_count = out_count;
  p.sets = static_cast<gsample::RowSet*>(workspace);
  try {
    if (R > 0) {
      st = launched(launch_sets((int)dtype, vec, R, most, &p, (cudaStream_t)stream));
      if (st != GSAMPLE_OK) return st;
    }
    // Eight CTAs a request at least: most draws are over in 3 us, and those from a
    // whole vocabulary are what the launch waits for.
    int c = fitting_cluster(gsample::verify_draw_kernel_fn((int)dtype, vec), false, n, most, p);
    const int64_t wide = (p.units_per_row + kUnitsPerCta - 1) / kUnitsPerCta;
    if (c < 8) c = wide < 8 ? (int)wide : 8;
    if (c > most) c = most;
    use_cluster(c, &p);
  } catch (...) {
    return GSAMPLE_ERR_CUDA;
  }
  return launched(gsample::launch_verify_draw(p, (int)dtype, vec, (cudaStream_t)stream));
}

gsample_status gsample_debug_weights(const float* x, int64_t n, float M, float T, uint64_t* out,
                                     gsample_stream_t stream) {
  if (n < 0 || !(T > 0.0f) || !std::isfinite(M) || (n > 0 && (!x || !out)) || misaligned(x, 4) ||
      misaligned(out, 8))
    return GSAMPLE_ERR_INVALID_ARG;
  if (n == 0) return GSAMPLE_OK;
  int sms = 0;
  const gsample_status st = gsample::current_device_sms(&sms);
  if (st != GSAMPLE_OK) return st;
  return launched(gsample::launch_debug_weights(x, n, M, T, out, (cudaStream_t)stream));
}

}  // extern "C"
