// Host side of the logit constraints: argument checks, launch planning and
// status mapping (include/gsample.h, "Logit constraints"). Nothing here touches
// device data or synchronises.
#include <climits>
#include <cstdint>
#include <cstring>

#include "gsample.h"
#include "gsample_internal.h"

namespace {

using gsample::ConstrainArgs;
using gsample::StateArgs;

constexpr int64_t kMaxV = (int64_t(1) << 31) - 128;

int64_t elt_bytes(gsample_dtype dt) { return dt == GSAMPLE_F32 ? 4 : 2; }

bool misaligned(const void* p, uintptr_t a) { return (uintptr_t)p % a != 0; }

gsample_status check_state(const gsample_logit_state* s, StateArgs* out) {
  if (!s || !s->history || !s->touched) return GSAMPLE_ERR_INVALID_ARG;
  if (misaligned(s->history, 16) || misaligned(s->bias, 16) || misaligned(s->touched, 4))
    return GSAMPLE_ERR_INVALID_ARG;
  if (s->rows < 1 || s->vocab < 1 || s->vocab > kMaxV || s->ld < s->vocab || s->ld % 32 != 0 ||
      s->ld > INT64_MAX / 4 / s->rows)
    return GSAMPLE_ERR_INVALID_ARG;
  out->history = reinterpret_cast<uint32_t*>(s->history);
  out->bias = s->bias;
  out->touched = s->touched;
  out->rows = s->rows;
  out->vocab = s->vocab;
  out->ld = s->ld;
  return GSAMPLE_OK;
}

gsample_status check_constraints(const gsample_constraints* c, int64_t B, int64_t V,
                                 ConstrainArgs* out) {
  std::memset(out, 0, sizeof *out);
  if (!c) return GSAMPLE_OK;
  if (c->state) {
    StateArgs s;
    const gsample_status st = check_state(c->state, &s);
    if (st != GSAMPLE_OK) return st;
    if (s.vocab != V || (!c->slot && s.rows < B)) return GSAMPLE_ERR_INVALID_ARG;
    if (misaligned(c->slot, 4) || misaligned(c->repetition, 4) || misaligned(c->frequency, 4) ||
        misaligned(c->presence, 4))
      return GSAMPLE_ERR_INVALID_ARG;
    out->history = s.history;
    out->bias = s.bias;
    out->touched = reinterpret_cast<const uint8_t*>(s.touched);
    out->state_rows = s.rows;
    out->state_ld = s.ld;
    out->slot = c->slot;
    out->repetition = c->repetition;
    out->frequency = c->frequency;
    out->presence = c->presence;
  }
  if (c->mask) {
    if (misaligned(c->mask, 4) || misaligned(c->mask_row, 4) || c->mask_rows < 0 ||
        c->mask_ld < (V + 31) / 32 || (!c->mask_row && c->mask_rows < B) ||
        c->mask_ld > INT64_MAX / 4 / (c->mask_rows > 0 ? c->mask_rows : 1))
      return GSAMPLE_ERR_INVALID_ARG;
    out->mask = reinterpret_cast<const uint8_t*>(c->mask);
    out->mask_rows = c->mask_rows;
    out->mask_ld_bytes = c->mask_ld * 4;
    out->mask_row = c->mask_row;
  }
  return GSAMPLE_OK;
}

gsample_status launched(cudaError_t e) {
  if (e == cudaSuccess) return GSAMPLE_OK;
  cudaGetLastError();
  return GSAMPLE_ERR_CUDA;
}

// Lists of n requests, `total` entries in all.
gsample_status check_lists(const int32_t* slot, int64_t n, const StateArgs& s,
                           const int64_t* tokens, int64_t total, const int64_t* offsets) {
  if (n < 0 || n > INT32_MAX || total < 0 || (!slot && n > s.rows)) return GSAMPLE_ERR_INVALID_ARG;
  if (!offsets && total != n) return GSAMPLE_ERR_INVALID_ARG;
  if (misaligned(slot, 4) || misaligned(tokens, 8) || misaligned(offsets, 8))
    return GSAMPLE_ERR_INVALID_ARG;
  if (total > 0 && !tokens) return GSAMPLE_ERR_INVALID_ARG;
  return GSAMPLE_OK;
}

// Whether some row of `out` shares a byte with some row of the logits. With
// one pitch for both the rows interleave, and only the spans within a pitch
// matter; otherwise the whole extents are compared.
bool rows_overlap(const char* x, int64_t x_row, int64_t x_ld, const char* y, int64_t y_row,
                  int64_t y_ld, int64_t B) {
  const uintptr_t x0 = (uintptr_t)x, y0 = (uintptr_t)y;
  const uintptr_t x1 = x0 + (uintptr_t)((B - 1) * x_ld + x_row);
  const uintptr_t y1 = y0 + (uintptr_t)((B - 1) * y_ld + y_row);
  if (x1 <= y0 || y1 <= x0) return false;
  if (x_ld != y_ld || B == 1) return true;
  const int64_t pitch = x_ld;
  int64_t d = (int64_t)(y0 > x0 ? (y0 - x0) % (uintptr_t)pitch : (x0 - y0) % (uintptr_t)pitch);
  if (y0 < x0 && d) d = pitch - d;  // start of y's span within x's pitch
  return !(d >= x_row && d + y_row <= pitch);
}

}  // namespace

extern "C" {

int64_t gsample_logit_state_ld(int64_t V) { return V > 0 ? (V + 31) / 32 * 32 : 0; }

gsample_status gsample_state_reset(const gsample_logit_state* state, const int32_t* slot,
                                   int64_t n, gsample_stream_t stream) {
  StateArgs s;
  gsample_status st = check_state(state, &s);
  if (st != GSAMPLE_OK) return st;
  st = check_lists(slot, n, s, nullptr, 0, reinterpret_cast<const int64_t*>(8));
  if (st != GSAMPLE_OK || n == 0) return st;
  int sms = 0;
  st = gsample::current_device_sms(&sms);
  if (st != GSAMPLE_OK) return st;
  return launched(gsample::launch_state_reset(s, slot, n, sms, (cudaStream_t)stream));
}

gsample_status gsample_history_append(const gsample_logit_state* state, const int32_t* slot,
                                      int64_t n, const int64_t* tokens, int64_t total,
                                      const int64_t* offsets, gsample_history_kind kind,
                                      gsample_stream_t stream) {
  StateArgs s;
  gsample_status st = check_state(state, &s);
  if (st != GSAMPLE_OK) return st;
  if (kind != GSAMPLE_HISTORY_PROMPT && kind != GSAMPLE_HISTORY_OUTPUT)
    return GSAMPLE_ERR_INVALID_ARG;
  st = check_lists(slot, n, s, tokens, total, offsets);
  if (st != GSAMPLE_OK || n == 0 || total == 0) return st;
  int sms = 0;
  st = gsample::current_device_sms(&sms);
  if (st != GSAMPLE_OK) return st;
  return launched(gsample::launch_history_append(s, slot, n, tokens, total, offsets,
                                                 kind == GSAMPLE_HISTORY_PROMPT, sms,
                                                 (cudaStream_t)stream));
}

gsample_status gsample_bias_set(const gsample_logit_state* state, const int32_t* slot, int64_t n,
                                const int64_t* tokens, const float* values, int64_t total,
                                const int64_t* offsets, gsample_stream_t stream) {
  StateArgs s;
  gsample_status st = check_state(state, &s);
  if (st != GSAMPLE_OK) return st;
  if (!s.bias || misaligned(values, 4)) return GSAMPLE_ERR_INVALID_ARG;
  st = check_lists(slot, n, s, tokens, total, offsets);
  if (st != GSAMPLE_OK || n == 0 || total == 0) return st;
  if (!values) return GSAMPLE_ERR_INVALID_ARG;
  int sms = 0;
  st = gsample::current_device_sms(&sms);
  if (st != GSAMPLE_OK) return st;
  return launched(gsample::launch_bias_set(s, slot, n, tokens, values, total, offsets,
                                           (cudaStream_t)stream));
}

gsample_status gsample_process_logits(const void* logits, gsample_dtype dtype, int64_t B,
                                      int64_t V, int64_t ld,
                                      const gsample_constraints* constraints, void* out,
                                      gsample_dtype out_dtype, int64_t out_ld,
                                      gsample_stream_t stream) {
  gsample_status st = gsample::check_logits(logits, dtype, B, V, ld);
  if (st != GSAMPLE_OK) return st;
  if (out_dtype != GSAMPLE_F32 && out_dtype != dtype) return GSAMPLE_ERR_INVALID_ARG;
  st = gsample::check_logits(out, out_dtype, B, V, out_ld);
  if (st != GSAMPLE_OK) return st;
  gsample::ProcessParams p;
  std::memset(&p, 0, sizeof p);
  st = check_constraints(constraints, B, V, &p.con);
  if (st != GSAMPLE_OK || B == 0) return st;
  p.logits = static_cast<const char*>(logits);
  p.out = static_cast<char*>(out);
  p.ld_bytes = ld * elt_bytes(dtype);
  p.out_ld_bytes = out_ld * elt_bytes(out_dtype);
  p.B = B;
  p.V = V;
  p.inplace = logits == out && dtype == out_dtype && (ld == out_ld || B == 1);
  if (!p.inplace && rows_overlap(p.logits, V * elt_bytes(dtype), p.ld_bytes, p.out,
                                 V * elt_bytes(out_dtype), p.out_ld_bytes, B))
    return GSAMPLE_ERR_INVALID_ARG;
  int sms = 0;
  st = gsample::current_device_sms(&sms);
  if (st != GSAMPLE_OK) return st;
  return launched(
      gsample::launch_process(p, (int)dtype, (int)out_dtype, sms, (cudaStream_t)stream));
}

gsample_status gsample_constrained_gumbel_argmax(const void* logits, gsample_dtype dtype,
                                                 int64_t B, int64_t V, int64_t ld,
                                                 const float* temperature, const uint64_t* seed,
                                                 const uint64_t* offset,
                                                 const gsample_constraints* constraints,
                                                 int64_t* out_idx, void* workspace,
                                                 gsample_stream_t stream) {
  if (B > 0 && (!temperature || !seed || !offset)) return GSAMPLE_ERR_INVALID_ARG;
  gsample_status st = gsample::check_logits(logits, dtype, B, V, ld);
  if (st != GSAMPLE_OK) return st;
  ConstrainArgs con;
  st = check_constraints(constraints, B, V, &con);
  if (st != GSAMPLE_OK) return st;
  try {  // launch plans are kept in a map, which may fail to grow
    return gsample::sample_constrained(logits, dtype, B, V, ld, temperature, seed, offset, con,
                                       out_idx, workspace, (cudaStream_t)stream);
  } catch (...) {
    return GSAMPLE_ERR_CUDA;
  }
}

}  // extern "C"
