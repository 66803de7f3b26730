/*
 * gsample -- batch Gumbel-max token sampling on GB300 (sm_103a).
 *
 * One launch samples one token per row of a [B, V] logits matrix. For every
 * element it forms
 *
 *     score_i = logits[i] / T + g_i,     g_i = -log(-log u_i),
 *
 * and returns the index of the largest score of each row. That index is an
 * exact sample of softmax(logits / T), with no softmax and no sort
 * ("Softmax-free GPU sampling: Gumbel-max categorical sampling kernel",
 * lablup/mlxcel issue #900, sections Background and Task 1). The uniform u_i
 * comes from a stateless Philox4x32-10 stream (Salmon et al., "Parallel Random
 * Numbers: As Easy as 1, 2, 3", SC'11) keyed by the row's 64-bit seed, with
 * counter (i >> 2, row, offset_lo32, offset_hi32); element i takes output word
 * i & 3; u_i = ((word >> 9) + 0.5) * 2^-23. Equal scores go to the lowest index.
 *
 * Conventions shared by every entry point:
 *   - logits: device pointer to B rows of V elements (dtype below); row b starts
 *     at element b * ld (ld >= V). Any element alignment is accepted; rows that
 *     start on a 16-byte boundary use 128-bit loads.
 *   - out_idx: device int64[B], written with the sampled index of each row, or
 *     -1 for a row with no candidate (every logit -inf or NaN).
 *   - NaN logits are never drawn; a +inf logit scores +inf (so the lowest +inf
 *     index of a row wins); scores are formed in binary32, where a finite logit
 *     whose quotient by T overflows scores +inf as well.
 *   - temperature / seed / offset: device arrays of B entries. A row whose
 *     temperature is <= 0 or NaN is sampled greedily (plain argmax of the raw
 *     logits, lowest index on ties), as the issue's Task 3 keeps greedy on argmax.
 *   - workspace: device buffer of gsample_workspace_bytes(B) bytes, zeroed once
 *     (gsample_workspace_init or a memset) before first use. Every launch that
 *     completes leaves it zeroed again, so it needs no clearing between calls.
 *     Two launches that are in flight at the same time (different streams) must
 *     not share a workspace.
 *   - stream: a cudaStream_t (NULL = legacy default stream). Calls only enqueue
 *     work on it and never synchronise; GSAMPLE_OK means "launched". Kernels are
 *     launched with programmatic stream serialization: each may be scheduled
 *     while the previous kernel of the stream drains, waits for it to complete
 *     before touching memory, and lets the next kernel be scheduled early. A
 *     kernel that follows on the stream with that launch attribute must wait
 *     (griddepcontrol.wait / cudaGridDependencySynchronize) before reading the
 *     indices; one launched without it sees the usual stream order.
 *   - The caller owns every buffer; the library allocates nothing and keeps no
 *     global state apart from cached device attributes.
 *   - Errors: arguments are checked on the host before anything is launched and
 *     a bad argument returns GSAMPLE_ERR_INVALID_ARG with nothing enqueued.
 *     Device data (temperatures, logits) is never validated. A launch failure
 *     returns GSAMPLE_ERR_CUDA. GSAMPLE_ERR_UNSUPPORTED means the current device
 *     is not a compute-capability 10.3 GPU.
 */
#ifndef GSAMPLE_H_
#define GSAMPLE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* gsample_stream_t;

typedef enum {
  GSAMPLE_F32 = 0,  /* IEEE binary32 */
  GSAMPLE_BF16 = 1, /* bfloat16, widened to binary32 exactly */
  GSAMPLE_F16 = 2   /* IEEE binary16, widened to binary32 exactly */
} gsample_dtype;

typedef enum {
  GSAMPLE_OK = 0,
  GSAMPLE_ERR_INVALID_ARG = 1,
  GSAMPLE_ERR_UNSUPPORTED = 2,
  GSAMPLE_ERR_WORKSPACE = 3,
  GSAMPLE_ERR_CUDA = 4
} gsample_status;

/* HLG pivot modes ("HLG sampling -- a piecewise tone curve on the logits",
 * section "The pivot"). */
typedef enum {
  GSAMPLE_PIVOT_TOP = 0,    /* mu = l_max - pivot_offset */
  GSAMPLE_PIVOT_ENTROPY = 1 /* mu = sum_i p_i l_i (minus the entropy) */
} gsample_pivot_mode;

/* HLG tone-curve parameters, in nats ("HLG sampling", sections "The transfer
 * function" and "Knobs"). With z = l - mu (l = log-softmax of the row):
 *   z < -w  : -m*w - m*beta_t*ln(1 + (-z - w)/beta_t)   (toe)
 *   |z| <= w:  m*z                                      (linear mid)
 *   z > w   :  m*w + m*beta_h*ln(1 + (z - w)/beta_h)    (shoulder)
 * Requirements: m > 0 finite; w >= 0 (w = +inf turns the rolloff off);
 * beta_t, beta_h > 0 finite; pivot_offset finite (used by the top mode). */
typedef struct {
  float m;
  float w;
  float beta_t;
  float beta_h;
  float pivot_offset;
  int32_t pivot_mode; /* gsample_pivot_mode */
} gsample_hlg_params;

/* Bytes of workspace needed for B rows (16 bytes per row). */
size_t gsample_workspace_bytes(int64_t B);

/* Zero the first gsample_workspace_bytes(B) bytes of `workspace` on `stream`. */
gsample_status gsample_workspace_init(void* workspace, int64_t B, gsample_stream_t stream);

/* Greedy decoding: out_idx[b] = lowest index of the largest logit of row b
 * (NaN and -inf never chosen; -1 if none). The issue keeps temperature 0 on a
 * plain argmax ("Softmax-free GPU sampling", Background and Task 3); the HLG
 * page's section "Greedy is untouched" says the same of the tone curve. */
gsample_status gsample_argmax(const void* logits, gsample_dtype dtype, int64_t B, int64_t V,
                              int64_t ld, int64_t* out_idx, void* workspace,
                              gsample_stream_t stream);

/* Gumbel-max sampling of every row in one launch ("Softmax-free GPU sampling",
 * Task 1: per-row RNG (seed, offset), temperature, batch-wide grid).
 * temperature[b] <= 0 or NaN selects greedy argmax for row b. */
gsample_status gsample_gumbel_argmax(const void* logits, gsample_dtype dtype, int64_t B,
                                     int64_t V, int64_t ld, const float* temperature,
                                     const uint64_t* seed, const uint64_t* offset,
                                     int64_t* out_idx, void* workspace,
                                     gsample_stream_t stream);

/* Top-k / top-p sampling on the Gumbel path, the follow-up "Softmax-free GPU
 * sampling" (Background) names as rejection-based top-k/top-p. Per row b the
 * filter set K is the first r candidates (logits that are neither NaN nor
 * -inf) in the order (logit descending, index ascending), where r is the
 * smaller of
 *   - top_k[b], when top_k[b] >= 1 (else no limit), and
 *   - the smallest prefix whose softmax(x / T) mass reaches top_p[b] * (row
 *     mass), when top_p[b] < 1 (top_p[b] <= 0 keeps the first candidate only;
 *     top_p[b] >= 1 or NaN: no limit);
 * and out_idx[b] is the Gumbel-max over K with the same noise as
 * gsample_gumbel_argmax: argmax over i in K of x_i / T + g_i, lowest index on
 * ties. It is an exact draw of softmax(x / T) restricted to K.
 *   - Rejection: the unfiltered draw (gsample_gumbel_argmax) is a proposal; a
 *     second pass over each filtered row keeps it when it lies in K (it is
 *     then the argmax over K); rejected rows are resolved exactly by a radix
 *     select of K's last element and the Gumbel-max over K. Three launches on
 *     `stream`, no host synchronisation.
 *   - top_k and top_p are device arrays of B entries (int32, float); either
 *     may be NULL (that filter off for every row). Both NULL: the same as
 *     gsample_gumbel_argmax.
 *   - Rows with temperature <= 0 or NaN are greedy (K always holds the top
 *     element). A row with a +inf logit returns its lowest +inf index.
 *   - The nucleus masses are binary32 sums on the GPU: a row whose top_p lands
 *     within ~1e-5 of the row mass from a prefix boundary may take one element
 *     more or less than an exact computation would.
 *   - Workspace, layout, validation and asynchrony as gsample_gumbel_argmax; a
 *     misaligned top_k/top_p (4 bytes) returns GSAMPLE_ERR_INVALID_ARG. */
gsample_status gsample_filtered_gumbel_argmax(const void* logits, gsample_dtype dtype, int64_t B,
                                              int64_t V, int64_t ld, const float* temperature,
                                              const uint64_t* seed, const uint64_t* offset,
                                              const int32_t* top_k, const float* top_p,
                                              int64_t* out_idx, void* workspace,
                                              gsample_stream_t stream);

/* HLG tone curve on the row's log-probs, then Gumbel-max ("HLG sampling",
 * sections "The transfer function", "The pivot", "Temperature semantics"):
 *     score_i = g(l_i - mu) / T + g_i,
 * where l = log_softmax(logits) and mu is the pivot of `hlg->pivot_mode`.
 * Dividing the curve by T is the pages' folding of temperature into the gain.
 * Rows with temperature <= 0 or NaN are greedy on the raw logits (the curve is
 * monotone, so it cannot move the argmax). `hlg` is a host pointer read during
 * the call. */
gsample_status gsample_hlg_gumbel_argmax(const void* logits, gsample_dtype dtype, int64_t B,
                                         int64_t V, int64_t ld, const float* temperature,
                                         const uint64_t* seed, const uint64_t* offset,
                                         const gsample_hlg_params* hlg, int64_t* out_idx,
                                         void* workspace, gsample_stream_t stream);

/* gsample_hlg_gumbel_argmax with one curve per row ("HLG sampling", section
 * "Where it lands in the code": each batched row owns its sampler, so the
 * curve parameters batch per request). hlg_rows: DEVICE array of B
 * gsample_hlg_params (24 bytes each, 4-byte aligned), read by the kernel.
 * Device data cannot be checked at the call, so a row whose parameters fail
 * the checks of gsample_hlg_gumbel_argmax (finite m > 0, w >= 0 (may be
 * +inf), finite beta_t > 0 and beta_h > 0, finite pivot_offset, a known
 * pivot_mode) gets out_idx[b] = -1; rows with temperature <= 0 or NaN are
 * greedy whatever their curve. Everything else as gsample_hlg_gumbel_argmax. */
gsample_status gsample_hlg_gumbel_argmax_rows(const void* logits, gsample_dtype dtype, int64_t B,
                                              int64_t V, int64_t ld, const float* temperature,
                                              const uint64_t* seed, const uint64_t* offset,
                                              const gsample_hlg_params* hlg_rows,
                                              int64_t* out_idx, void* workspace,
                                              gsample_stream_t stream);

/* The categorical baseline the issue measures Gumbel-max against ("Softmax-free
 * GPU sampling", Background and Performance validation): a normalisation of
 * softmax(logits / T) and one inverse-CDF draw per row,
 *     out_idx[b] = smallest i with e_0 + ... + e_i > u * S,
 * e_i = exp((x_i - M) / T) (0 for -inf and NaN), M the largest finite logit,
 * S = sum e_i, u the uniform of element 0's Philox word of the row's
 * (seed, offset) stream (the same word gsample_gumbel_argmax gives element 0).
 * temperature <= 0 or NaN is greedy; a +inf logit takes all the mass (lowest
 * +inf index); -1 if the row has no candidate. The sums are binary32: the
 * index is the inverse CDF of a target within about 1e-6 of S of u * S (not
 * bit-exact against a double-precision CDF). Needs no workspace. Device
 * pointers, caller stream, asynchronous, host-side validation as above. */
gsample_status gsample_categorical(const void* logits, gsample_dtype dtype, int64_t B, int64_t V,
                                   int64_t ld, const float* temperature, const uint64_t* seed,
                                   const uint64_t* offset, int64_t* out_idx,
                                   gsample_stream_t stream);

/* Static, human-readable name of a status code. */
const char* gsample_status_string(gsample_status status);

/* Largest batch gsample_gumbel_argmax_static accepts. */
#define GSAMPLE_STATIC_WS_MAX_ROWS 4096

/* gsample_gumbel_argmax without a workspace argument: the merge state lives in
 * a fixed array inside the library (GSAMPLE_STATIC_WS_MAX_ROWS rows, 64 KiB),
 * so the call allocates no device memory. The source pages have no counterpart
 * to this entry point; it exists for callers that cannot allocate: code that
 * runs inside a host framework or engine plugin which owns all device memory
 * and forbids allocations while it executes, code with a device-memory budget
 * fixed at start-up, and decode loops where cudaMalloc/cudaFree would stall the
 * GPU with their implicit synchronisation.
 *   - The caller still passes the inputs and out_idx (same meaning as in
 *     gsample_gumbel_argmax); B > GSAMPLE_STATIC_WS_MAX_ROWS returns
 *     GSAMPLE_ERR_INVALID_ARG with nothing enqueued; B == 0 is a no-op.
 *   - Every other argument is checked as gsample_gumbel_argmax checks it, and
 *     a bad one returns that entry point's status with nothing enqueued.
 *   - The array is held by every GPU that loads the library until the process
 *     exits, and is zero when the library's device code loads. The first call
 *     on each device looks up its device address (cudaGetSymbolAddress) and
 *     keeps it for the life of the process: do not call this entry point again
 *     on a device after cudaDeviceReset. That first call must not be made while
 *     `stream` is being captured: it returns GSAMPLE_ERR_UNSUPPORTED, with
 *     nothing enqueued. A failed look-up returns GSAMPLE_ERR_CUDA.
 *   - Every call clears the rows it uses (an asynchronous memset on `stream`)
 *     before sampling, and calls no cudaMalloc, cudaFree or other allocating
 *     routine.
 *   - All calls on a device share the one array: calls whose work overlaps on
 *     the GPU (different streams, or host threads racing) race on it and may
 *     return wrong indices. Serialise them, for example on one stream. */
gsample_status gsample_gumbel_argmax_static(const void* logits, gsample_dtype dtype, int64_t B,
                                            int64_t V, int64_t ld, const float* temperature,
                                            const uint64_t* seed, const uint64_t* offset,
                                            int64_t* out_idx, gsample_stream_t stream);

/* gsample_gumbel_argmax on host-resident data, with no staging copy: logits,
 * temperature, seed, offset and out_idx are page-locked HOST buffers
 * (cudaHostAlloc / cudaMallocHost, or cudaHostRegister), which the kernel
 * reads and writes through their mapping into the current device. On a GB300
 * the loads cross the CPU-GPU link once per logit; no device copy of the
 * logits is made. workspace stays a DEVICE buffer.
 *   - Each of the five host pointers is looked up with cudaPointerGetAttributes.
 *     One that is not page-locked host memory mapped into the current device
 *     returns GSAMPLE_ERR_INVALID_ARG, a workspace that is not device memory
 *     GSAMPLE_ERR_WORKSPACE; nothing is enqueued in either case. Buffer sizes
 *     cannot be checked: the caller guarantees B rows of ld elements, and B
 *     entries of the per-row arrays.
 *   - Asynchronous on `stream`: out_idx holds the indices once `stream` has been
 *     synchronised, and the host must not write the inputs before then.
 *   - Shapes, ld, alignment, NaN/inf handling, greedy rows and the workspace
 *     contract are those of gsample_gumbel_argmax, and so are the indices.
 *   - Its rate is the link's (host-to-device reads measured about 0.21 TB/s on
 *     GB300, the same as cudaMemcpyAsync), not the kernel's. */
gsample_status gsample_gumbel_argmax_host(const void* logits, gsample_dtype dtype, int64_t B,
                                          int64_t V, int64_t ld, const float* temperature,
                                          const uint64_t* seed, const uint64_t* offset,
                                          int64_t* out_idx, void* workspace,
                                          gsample_stream_t stream);

/* ---------------------------------------------------------------------------
 * Logit constraints: the steps between a model's logits and the draw that
 * "Softmax-free GPU sampling" (Background) lists ahead of the sampler: token
 * bias and repetition / frequency / presence penalties, and grammar masks.
 *
 * For element v of row b, with x = logits[b, v] in binary32, the state row r
 * and the row's parameters, the constrained logit is
 *
 *   if x == -inf:               -inf (a token masked upstream stays masked)
 *   otherwise                   x = x + bias[r, v]
 *     if history[r, v] != 0:    x = x > 0 ? x / repetition : x * repetition
 *     with c = history & 0x7fffffff, if c > 0:
 *                               x = (x - frequency * c) - presence
 *   if the mask bit of v is 0:  -inf, whatever x is (NaN and +inf included)
 *
 * each operation rounded once to binary32. A repetition that is not finite or
 * not > 0 counts as 1, a NaN frequency or presence as 0.
 * ------------------------------------------------------------------------- */

/* What each request has seen and the biases it asked for, on the device: the
 * caller owns the three arrays, zeroes them once, and passes this struct (host
 * memory, read during the call). State rows are a server's request slots; a
 * batch row picks its own through `slot`.
 *   history  int32 [rows, ld]: bits 0..30 count the token's appearances in the
 *            output so far; bit 31 is set when it is in the prompt. The
 *            repetition penalty applies to both, frequency and presence to the
 *            output alone.
 *   bias     float [rows, ld], or NULL: no biases.
 *   touched  uint32 [rows, ld / 32]: bit v & 31 of word v >> 5 is set where
 *            history or bias may be nonzero; entries without it hold zeros. The
 *            calls below keep it so.
 *   rows >= 1; vocab = V of the logits; ld a multiple of 32, >= vocab
 *   (gsample_logit_state_ld). history and bias are 16-byte aligned, touched
 *   4-byte aligned.
 * A token may be counted up to 2^31 - 1 times.
 * The layout is public: rows may be copied (a forked request), saved and
 * restored by plain copies of the three arrays. Calls that write a state must
 * be ordered (by stream or event) with every call that uses it. */
typedef struct {
  int32_t* history;
  float* bias;
  uint32_t* touched;
  int64_t rows;
  int64_t vocab;
  int64_t ld;
} gsample_logit_state;

/* The constraints of a batch (host memory, read during the call; the arrays
 * are device memory). Any part may be absent (NULL).
 *   state       penalties and biases; NULL: neither.
 *   slot        int32[B]: the state row of each batch row; a value outside
 *               [0, rows) means no state for that row. NULL: row b uses state
 *               row b (rows >= B).
 *   repetition, frequency, presence   float[B]; NULL: 1, 0, 0.
 *   mask        packed masks [mask_rows, mask_ld] of 32-bit words, bit v & 31
 *               of word v >> 5 set where token v is allowed; mask_ld words
 *               (>= ceil(V / 32)) from row to row. Bits at and past V are
 *               ignored. 4-byte aligned.
 *   mask_row    int32[B]: the mask row of each batch row; a value outside
 *               [0, mask_rows) means no mask. NULL: row b uses mask row b
 *               (mask_rows >= B). */
typedef struct {
  const gsample_logit_state* state;
  const int32_t* slot;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const uint32_t* mask;
  int64_t mask_rows;
  int64_t mask_ld;
  const int32_t* mask_row;
} gsample_constraints;

/* Which part of the history gsample_history_append extends. */
typedef enum {
  GSAMPLE_HISTORY_PROMPT = 0, /* sets bit 31 */
  GSAMPLE_HISTORY_OUTPUT = 1  /* adds one to the count */
} gsample_history_kind;

/* Smallest ld of a state for vocabulary V: V rounded up to a multiple of 32. */
int64_t gsample_logit_state_ld(int64_t V);

/* Clears n state rows (history, bias and touched bits): those in slot[0..n)
 * (device int32, values outside [0, rows) ignored), or the first n when slot
 * is NULL. Reads the touched bits and writes only what they mark. */
gsample_status gsample_state_reset(const gsample_logit_state* state, const int32_t* slot,
                                   int64_t n, gsample_stream_t stream);

/* Appends tokens to the history of n requests. Request i owns
 * tokens[offsets[i] .. offsets[i + 1]) (device int64, offsets[0..n] not
 * decreasing; positions outside [0, total) and outside every request are
 * ignored), or tokens[i] alone when offsets is NULL (total == n: the indices a
 * sampler just drew, say). slot as in gsample_state_reset. Token ids outside
 * [0, vocab) are ignored (a sampler's -1 too). A slot or a token may appear
 * more than once: every appearance counts. */
gsample_status gsample_history_append(const gsample_logit_state* state, const int32_t* slot,
                                      int64_t n, const int64_t* tokens, int64_t total,
                                      const int64_t* offsets, gsample_history_kind kind,
                                      gsample_stream_t stream);

/* Sets bias[slot, tokens[j]] = values[j] for the lists of n requests (layout
 * as in gsample_history_append). Other entries keep their values. A token
 * named twice in one list takes the later value; a slot named by two requests
 * of one call takes either request's value. A list is walked in order by one
 * warp: 4 us for 300 entries, 29 us for 3000, 0.9 ms for 100000.
 * state->bias must not be NULL. */
gsample_status gsample_bias_set(const gsample_logit_state* state, const int32_t* slot, int64_t n,
                                const int64_t* tokens, const float* values, int64_t total,
                                const int64_t* offsets, gsample_stream_t stream);

/* Writes the constrained logits of every row: out[b, v], rounded once to
 * out_dtype, which is GSAMPLE_F32 or the logits' type; out_ld elements from
 * row to row. In place (out == logits, same type and ld) the elements that
 * change are written, and with them, unchanged, others near them: all of a run of
 * 32 elements, or of 16 bytes, of which the mask takes a part, and every element
 * whose touched bit is set. So nothing else may write the rows meanwhile. Any
 * other overlap of a row of out with a row of the logits returns
 * GSAMPLE_ERR_INVALID_ARG. constraints == NULL converts. */
gsample_status gsample_process_logits(const void* logits, gsample_dtype dtype, int64_t B,
                                      int64_t V, int64_t ld,
                                      const gsample_constraints* constraints, void* out,
                                      gsample_dtype out_dtype, int64_t out_ld,
                                      gsample_stream_t stream);

/* gsample_gumbel_argmax on the constrained logits, which are not written
 * anywhere and not rounded below binary32: the indices are those of
 * gsample_process_logits with GSAMPLE_F32 followed by gsample_gumbel_argmax.
 * A row whose mask leaves nothing gets -1; a constrained logit that is NaN
 * (a NaN bias, +inf less +inf) is never drawn. One or two launches. Everything
 * else (greedy rows, workspace, validation, asynchrony) as
 * gsample_gumbel_argmax. */
gsample_status gsample_constrained_gumbel_argmax(const void* logits, gsample_dtype dtype,
                                                 int64_t B, int64_t V, int64_t ld,
                                                 const float* temperature, const uint64_t* seed,
                                                 const uint64_t* offset,
                                                 const gsample_constraints* constraints,
                                                 int64_t* out_idx, void* workspace,
                                                 gsample_stream_t stream);

/* ---------------------------------------------------------------------------
 * Draws from given random numbers: the sampler of the issue's categorical path
 * ("Softmax-free GPU sampling", Background: temperature, top-k, top-p, min-p,
 * then a categorical draw) for callers that bring their own random numbers,
 * and the verification of speculative drafts by the same filter.
 * ------------------------------------------------------------------------- */

/* One draw a row from softmax(logits / T) restricted to the row's filter set K
 * by the inverse CDF in index order: out_idx[b] is the smallest i in K with
 *     sum of e_j over j <= i in K  >  u_b * (sum of e_j over K),
 * e_j = exp((x_j - M) / T), M the largest logit. K is the first r candidates
 * (logits that are neither NaN nor -inf) in the order (logit descending, index
 * ascending), r the smallest of
 *   - top_k[b], when top_k[b] >= 1 (else no limit),
 *   - the smallest prefix whose softmax mass reaches top_p[b] * (row mass),
 *     when top_p[b] < 1 (top_p[b] <= 0 keeps the first candidate only; >= 1 or
 *     NaN: no limit),
 *   - the elements with e_j >= min_p[b], when min_p[b] > 0 (above 1 counts as
 *     1; <= 0 or NaN: no limit),
 * and holds at least the first candidate.
 *   - uniform: device array of B floats in [0, 1) (below, or NaN: 0; 1 and
 *     above: the largest below 1). top_k, top_p, min_p: device arrays of B
 *     entries; any may be NULL (that filter off).
 *   - out_logprob: device float[B] or NULL: log(e_i / sum over K) of the drawn
 *     token, natural, rounded once (without a filter it may be off by 2^-24 before
 *     that); 0 for greedy rows, -inf for a row without candidates (out_idx -1).
 *   - T <= 0 or NaN: greedy. +inf logits: the lowest such index. T = +inf: all
 *     candidates weigh the same. Temperatures below 2^-126 count as that.
 *   - Weights are fixed-point numbers with 44 fraction bits (fewer past V =
 *     2^18), each within about 2^-39 of itself; their sums are exact and the
 *     result does not depend on the launch. So an index differs from the exact
 *     one only where u or a filter's border lies within about 1e-11 of the mass
 *     from a boundary. An element whose weight is below 2^-45 is never drawn.
 *   - Layout, alignment, errors and asynchrony as gsample_gumbel_argmax; B up
 *     to (2^31 - 1) / 16. No workspace. One or two launches (between them out_idx
 *     holds negative marks). */
gsample_status gsample_filtered_categorical(const void* logits, gsample_dtype dtype, int64_t B,
                                            int64_t V, int64_t ld, const float* temperature,
                                            const float* uniform, const int32_t* top_k,
                                            const float* top_p, const float* min_p,
                                            int64_t* out_idx, float* out_logprob,
                                            gsample_stream_t stream);

/* Bytes of workspace gsample_verify_drafts needs for R rows (32 a row; need not
 * be cleared). */
size_t gsample_verify_workspace_bytes(int64_t R);

/* Verification of the draft tokens of n requests against the target model's
 * logits, so that the tokens that come out are distributed as the target's own
 * draws. Request i owns rows offsets[i] .. offsets[i + 1] of the logits (device
 * int64, offsets[0..n] not decreasing, clipped to [0, R]): row r holds the
 * target's logits after the tokens up to draft[r - 1], draft[r] (device
 * int64[R]) is the token proposed next, and the request's last row has no draft
 * (its entry is ignored). p_r is softmax(logits / T) over the row's filter set,
 * normalised, as gsample_filtered_categorical has it, with the settings of
 * request i (temperature, top_k, top_p, min_p: device arrays of n entries).
 *   - draft_probs: device float rows (draft_probs_ld >= V elements from row to
 *     row), row r the distribution q_r that draft[r] was drawn from; NaN and
 *     negative entries count as 0, in the residual those above 1 as 1. The rows
 *     of last rows are not read. NULL: drafts without probabilities (looked up,
 *     or greedy), q_r(t) = 1 for the draft alone.
 *   - In order, draft[r] is accepted when uniform[r] * q_r(t) < p_r(t) (so a
 *     token outside [0, V) or outside the filter set is not). At the first
 *     that is not, the next token is drawn from max(p_r - q_r, 0), normalised
 *     (from p_r where that is zero everywhere); when all are, from p of the last
 *     row. uniform: device float[R]; uniform_draw: device float[n], the number
 *     of the request's one draw, which is the inverse CDF in index order.
 *   - out_tokens: device int64[R]. The rows of a request get its accepted
 *     drafts, then the drawn token, then -1 (also in place of a draw from a row
 *     without candidates): lists that gsample_history_append takes with the
 *     same offsets. Rows outside every request are left as they were.
 *   - out_count: device int32[n], the tokens a request got (0 for a request
 *     without rows).
 *   - workspace: device buffer of gsample_verify_workspace_bytes(R) bytes,
 *     16-byte aligned, with any contents; launches in flight at the same time
 *     must not share one. Two or three launches.
 * Temperatures <= 0, special values, precision, layout, validation and
 * asynchrony as gsample_filtered_categorical; R and n up to (2^31 - 1) / 16. */
gsample_status gsample_verify_drafts(const void* logits, gsample_dtype dtype, int64_t R, int64_t V,
                                     int64_t ld, int64_t n, const int64_t* offsets,
                                     const int64_t* draft, const float* draft_probs,
                                     int64_t draft_probs_ld, const float* temperature,
                                     const int32_t* top_k, const float* top_p, const float* min_p,
                                     const float* uniform, const float* uniform_draw,
                                     int64_t* out_tokens, int32_t* out_count, void* workspace,
                                     gsample_stream_t stream);

/* ---------------------------------------------------------------------------
 * Pages of a paged cache: the block tables and slot maps that the model's next
 * step needs, built where the number of accepted tokens is known.
 * ------------------------------------------------------------------------- */

/* Which physical pages hold the tokens of each request slot (the caller owns
 * the arrays; this struct is host memory, read during the call).
 *   table       int32 [rows, ld]: entry c of a slot is the page of its tokens
 *               c * page_size .. (c + 1) * page_size, -1 past its last page.
 *   length      int32 [rows]: tokens of each slot.
 *   free_list   int32 [pages]: a stack of free page ids; free_count int32[1]:
 *               how many it holds (the top is free_list[free_count - 1]).
 *   rows from 1 to 65536; ld * page_size, the longest slot, below 2^31.
 * To begin: table -1, length 0, free_list a permutation of the page ids and
 * free_count = pages. Page ids are the caller's: the library only moves them.
 * Calls that write a state must be ordered with every call that uses it. */
typedef struct {
  int32_t* table;
  int32_t* length;
  int32_t* free_list;
  int32_t* free_count;
  int64_t rows;
  int64_t ld;
  int64_t pages;
  int32_t page_size;
} gsample_page_state;

/* Appends room for tokens to n slots and builds what a model step over those
 * tokens needs. Request i appends the tokens offsets[i] .. offsets[i + 1]
 * (device int64, offsets[0..n] not decreasing, clipped to [0, total]), or one
 * token when offsets is NULL (total == n), to the slot slot[i] (device int32;
 * NULL: slot i). New pages come off the stack in order of i, lowest token first.
 *   - A request is refused, its slot left as it was, when its slot is outside
 *     [0, rows) or named by more than one request of the call, when it would
 *     pass ld * page_size tokens, or when it needs pages and those that it and
 *     the requests before it need (refused for want of pages or not) are more
 *     than the stack holds. A request that needs no new page is never refused
 *     for want of pages.
 *   - out_start: device int32[n], the length before (the position of the first
 *     new token), -1 for a refused request.
 *   - out_slot_map: device int64[total]: page * page_size + place in the page
 *     of each new token, -1 for those of a refused request; entries outside
 *     every request are left as they were.
 *   - out_length: device int32[n] or NULL: the length after, 0 where refused.
 *   - out_table: device int32 rows (table_ld >= table_cols entries from row to
 *     row) or NULL: the first table_cols entries of each request's table after
 *     the call, -1 past its last page and where refused. */
gsample_status gsample_pages_extend(const gsample_page_state* state, const int32_t* slot,
                                    int64_t n, const int64_t* offsets, int64_t total,
                                    int32_t* out_start, int64_t* out_slot_map, int32_t* out_length,
                                    int32_t* out_table, int64_t table_cols, int64_t table_ld,
                                    gsample_stream_t stream);

/* Shortens n slots to start[i] + keep[i] tokens (device int32; NULL counts as
 * 0, so both NULL release the slots), at least 0, and puts the pages past that
 * back on the stack, where an extension of the same requests takes them from in
 * the same order. A slot that is no longer, one outside [0, rows), one named
 * more than once in the call and one with a negative start (a request that
 * gsample_pages_extend refused) are left as they were. After a verification:
 * start from gsample_pages_extend, keep = out_count of gsample_verify_drafts. */
gsample_status gsample_pages_trim(const gsample_page_state* state, const int32_t* slot, int64_t n,
                                  const int32_t* start, const int32_t* keep,
                                  gsample_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GSAMPLE_H_ */
