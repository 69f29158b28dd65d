/*
 * ola.h — C ABI of the beam-parallel Gated DeltaNet decode library (sm_100a).
 *
 * What the library computes
 * -------------------------
 * One GDN layer of R requests x H heads. Every request decodes B beams that all start from
 * one shared post-prefill state S_ctx (d_v x d_k per request and head). Decode step t of new
 * beam b continues parent beam p = parent_idx[r][b] of step t-1 ("Scientific Impact
 * Assessment: OneLA", §1 Core Contribution: hundreds of beams start from one prompt-derived
 * state and diverge through a few decode-time transitions; pruning, reordering and fan-out
 * are expressed by the ancestry index). The transition is the gated delta rule (Gated Delta
 * Networks, listed under "Builds on" on the OneLA listing):
 *
 *     S_t = alpha_t * S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,   alpha_t = exp(g_t)
 *     o_t = S_t q_t
 *
 * The default (replay) path never forms a per-beam state. Each beam appends a transition
 * record (w_t, k_t, alpha_t) with u_t = S_{t-1} k_t and w_t = beta_t (v_t - alpha_t u_t), so
 * that S_t = alpha_t S_{t-1} + w_t k_t^T, and S_{t-1} x is evaluated as
 *     (prod alpha) S_ctx x + sum_j (prod_{i>j} alpha_i) w_j (k_j . x)
 * over the records of the beam's chain ("Scientific Impact Assessment: OneLA", §1: append-only
 * records of O(d_v + d_k) per beam, projection replay through the key and query
 * contractions, one kernel reusing S_ctx across beams; the OneLA listing's Abstract: records
 * are never moved or copied when beams are updated). Two comparison paths implement the
 * practices the Abstract contrasts with: FullState keeps one d_v x d_k state per beam, and the
 * history-replay path (REPLAYSSM) keeps no state at all and rebuilds every beam's state from
 * S_ctx over its chain's raw tokens at every step.
 *
 * Conventions (every entry point)
 * -------------------------------
 * - Tensors are row-major, contiguous, on the current CUDA device unless a function says
 *   "host". Layouts are given in brackets, slowest index first.
 * - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream). Calls are
 *   stream-ordered and asynchronous unless stated; inputs are borrowed only until the work
 *   queued on `stream` has run; the library never keeps a caller pointer.
 * - Host-side validation failures return at once, with nothing launched and no state changed.
 * - Device-side errors (an out-of-range parent, a bounded wait that ran out) are sticky: the
 *   kernel clamps and carries on and records the first code in a device word. ola_get_error
 *   waits for the handle's queued work and returns it; from then on ola_step refuses to run
 *   (returns that code, launches nothing) until ola_reset clears it. Outputs of a step that
 *   recorded an error are unspecified.
 * - A handle is used by one host thread at a time.
 * - Pointers to q, k, v, out_o and S_ctx must be 16-byte aligned; g, beta, parent_idx
 *   4-byte aligned.
 */
#ifndef OLA_H_
#define OLA_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  OLA_OK = 0,
  OLA_ERR_INVALID_ARG = 1,   /* NULL / misaligned pointer, bad size, bad enum */
  OLA_ERR_UNSUPPORTED = 2,   /* geometry outside what this build supports, or not sm_100 */
  OLA_ERR_CAPACITY = 3,      /* ola_step after T_max steps (nothing launched) */
  OLA_ERR_BAD_PARENT = 4,    /* a parent index was out of range (device-detected, sticky) */
  OLA_ERR_OOM = 5,           /* device allocation failed */
  OLA_ERR_CUDA = 6,          /* a CUDA runtime call failed */
  OLA_ERR_TIMEOUT = 7,       /* a bounded device wait ran out (device-detected, sticky) */
  OLA_ERR_SCRATCH_LIMIT = 8  /* ola_decode_noalloc: problem larger than its fixed scratch */
} ola_status;

/* dtype of q, k, v (and of the prompt's k, v for ola_prefill) */
enum { OLA_F32 = 0, OLA_BF16 = 1 };
/* how beam states are represented:
 * REPLAY     = one shared state + append-only transition records (w, k, alpha) per beam,
 *              evaluated by projection replay (the method);
 * FULLSTATE  = one materialised d_v x d_k fp32 state per beam, ping-pong buffers (comparison);
 * REPLAYSSM  = no per-beam state kept: each step rebuilds every beam's state from the shared
 *              state by replaying the raw tokens (k, v, alpha, beta) on its chain, fp32
 *              (comparison). */
enum { OLA_PATH_REPLAY = 0, OLA_PATH_FULLSTATE = 1, OLA_PATH_REPLAYSSM = 2 };
/* how the contractions of the replay path are computed:
 * FP32 = CUDA-core fp32 FMA everywhere; TENSOR = tcgen05 tensor cores, bf16 operands with
 * S_ctx split into a bf16 high part and a bf16 remainder (two MMAs, fp32 accumulate in
 * tensor memory). With B <= 1024 and T_max <= 12 the replay accumulation over the ancestor
 * records also runs on tensor cores: the records' w rows are then kept as a bf16 high part and
 * a bf16 remainder (same bytes as fp32) and each product runs as three bf16 MMAs with fp32
 * accumulation; beyond those limits it runs in fp32 on CUDA cores. */
enum { OLA_MATH_FP32 = 0, OLA_MATH_TENSOR = 1 };

typedef struct {
  int32_t R;          /* requests, >= 1 */
  int32_t H;          /* heads, >= 1 */
  int32_t d_k;        /* key width: 16, 32, 64, 128 or 256 (TENSOR: 64, 128, 256) */
  int32_t d_v;        /* value width: 16, 32, 64, 128 or 256 (TENSOR: 64, 128, 256) */
  int32_t B;          /* beams per request, 1..4096 (TENSOR: T_max*R*H*B < 2^31) */
  int32_t T_max;      /* decode steps the handle can hold, 1..32 */
  int32_t in_dtype;   /* OLA_F32 or OLA_BF16 (TENSOR: OLA_BF16) */
  int32_t path;       /* OLA_PATH_REPLAY, OLA_PATH_FULLSTATE or OLA_PATH_REPLAYSSM */
  int32_t math;       /* OLA_MATH_FP32 or OLA_MATH_TENSOR (replay path only) */
} ola_geometry;

typedef struct ola_ctx* ola_handle;

/* Library version, (major << 16) | minor. Never fails, touches no device. */
int32_t ola_version(void);

/* Static message for a status code. Never fails, touches no device. */
const char* ola_strerror(ola_status s);

/* Device bytes a handle of this geometry will own (records, ancestry, state copies).
 * Host-only; validates like ola_create. */
ola_status ola_workspace_bytes(const ola_geometry* geom, uint64_t* out_bytes);

/* Create a decoder for one GDN layer of R requests.
 *   geom   : host pointer, copied.
 *   S_ctx  : device [R][H][d_v][d_k] fp32, the shared post-prefill state of each (request,
 *            head). Copied into the handle on `stream`; the caller may free it once the stream
 *            has reached this point.
 *   out    : host pointer that receives the handle (set to NULL on failure).
 * Allocates every buffer of ola_workspace_bytes on the current device. Step counter t = 0.
 * Errors: INVALID_ARG, UNSUPPORTED (geometry, or device is not sm_100), OOM, CUDA. */
ola_status ola_create(const ola_geometry* geom, const float* S_ctx, void* stream,
                      ola_handle* out);

/* One decode step (t := t + 1) for every request, beam and head.
 *   q, k       : device [R][B][H][d_k], in_dtype. q, k are used as given (no normalisation,
 *                no scaling).
 *   v          : device [R][B][H][d_v], in_dtype.
 *   g          : device [R][B][H] fp32, log decay (alpha = exp(g)).
 *   beta       : device [R][B][H] fp32, write strength.
 *   parent_idx : device [R][B] int32. Step 1: must be 0 (the shared state is the only
 *                parent). Later steps: index of the parent beam among the previous step's B
 *                beams, shared by all heads of the request. Out of range: clamped to 0 and
 *                OLA_ERR_BAD_PARENT is recorded (sticky).
 *   out_o      : device [R][B][H][d_v] fp32, o_t = S_t q_t (written, never read).
 * Errors: INVALID_ARG, CAPACITY (t == T_max; nothing launched), a sticky device error that
 * ola_get_error has returned (nothing launched), CUDA. */
ola_status ola_step(ola_handle h, const void* q, const void* k, const void* v, const float* g,
                    const float* beta, const int32_t* parent_idx, float* out_o, void* stream);

/* ola_step with HOST buffers of the same layouts: copies the inputs into library-owned
 * device staging buffers (one cudaMemcpyAsync per tensor), runs the step, copies out_o
 * back, and returns after `stream` has finished (synchronous). Pinned host memory makes
 * the copies asynchronous DMA; pageable memory works but is slower. */
ola_status ola_step_host(ola_handle h, const void* q, const void* k, const void* v,
                         const float* g, const float* beta, const int32_t* parent_idx,
                         float* out_o, void* stream);

/* ola_step_host without waiting: pipelined decode from host buffers. The inputs are copied
 * in on a copy stream of the handle, the step runs on `stream` and out_o is copied back on a
 * second copy stream, so one call's copy-out overlaps the next call's copy-in (the host link
 * carries both directions at once). Two device staging sets are used in turn. Returns once the
 * work is queued. The host buffers of a call must stay valid, and out_o unread, until
 * ola_host_sync; they must be pinned for the copies to be asynchronous.
 * Errors: as ola_step; INVALID_ARG for NULL pointers; CUDA. */
ola_status ola_step_host_async(ola_handle h, const void* q, const void* k, const void* v,
                               const float* g, const float* beta, const int32_t* parent_idx,
                               float* out_o, void* stream);

/* Wait for every queued ola_step_host_async call (its copies and steps); then as
 * ola_get_error. */
ola_status ola_host_sync(ola_handle h);

/* Rewind to t = 0, keeping S_ctx, and clear the sticky device error. Stream-ordered on the
 * stream of the handle's last call (no host synchronisation): work queued before it still
 * runs, and the next ola_step must be queued on that stream or ordered after it. */
ola_status ola_reset(ola_handle h);

/* Current step t (0 .. T_max), or -1 for a NULL handle. Host-only. */
int32_t ola_current_step(ola_handle h);

/* Ancestry of the current beams: out[r][b][s] (device [R][B][t] int32) = the beam index of
 * the record that beam b's chain holds at step s+1 (out[r][b][t-1] == b). Stream-ordered.
 * Errors: INVALID_ARG (NULL, or t == 0), CUDA. */
ola_status ola_get_ancestry(ola_handle h, int32_t* out, void* stream);

/* Wait for the handle's queued work, then return its sticky device error (OLA_OK if none). */
ola_status ola_get_error(ola_handle h);

/* Record reclamation ("Scientific Impact Assessment: OneLA", §1: append-only transition
 * records over one shared post-prefill state, pruning through the parent-pointer ancestry
 * index). Finds the longest prefix of chain slots at which every live beam of every request
 * holds the same record (beam search that has converged), folds those records into S_ctx in
 * chain order (S <- alpha_j S + w_j k_j^T, the transition written with the record; fp32, and
 * the bf16 split of the tensor path is recomputed), moves the later records, chain rows and
 * ranks down by that many slots and decreases t by it. Later steps give the same outputs up to
 * rounding, and a decode can run past T_max while its beams keep converging. The current
 * step's own records are never folded (t stays >= 1). ola_get_ancestry afterwards returns the
 * chains without the folded slots, and ola_reset keeps the folded S_ctx. On the REPLAYSSM
 * path the folded records are raw tokens and are applied with the gated delta rule itself.
 *   out_folded : host int32, optional (NULL): number of folded steps (0 if none).
 * Synchronises `stream`, which must be the stream of the handle's previous calls (or ordered
 * after them). FullState handles keep every beam's state, so nothing is folded there: only the
 * ancestry rows of the shared slots are dropped and t lowered, which lets them decode past T_max
 * too (out_folded counts those slots).
 * Errors: INVALID_ARG (NULL handle), the sticky device error, CUDA. */
ola_status ola_compact(ola_handle h, int32_t* out_folded, void* stream);

/* Free every buffer of the handle (waits for its queued work first). NULL is a no-op.
 * The handle must not be used afterwards. */
ola_status ola_destroy(ola_handle h);

/* Shared post-prefill state from a prompt: for each (request, head), start from S = 0 and
 * apply the transition above to the prompt tokens p = 0..P-1 in order ("Scientific Impact
 * Assessment: OneLA", §1: one state derived from the shared prompt), in fp32.
 *   k    : device [R][P][H][d_k], in_dtype;   v : device [R][P][H][d_v], in_dtype
 *   g    : device [R][P][H] fp32 (log decay);  beta : device [R][P][H] fp32
 *   S_out: device [R][H][d_v][d_k] fp32 (written).
 * d_k, d_v in {16, 32, 64, 128, 256}; P >= 0 (P = 0 writes zeros).
 * d_k = d_v = 128 with a bf16 prompt (k, v 16-byte aligned) runs the chunked tensor-core form
 * (64 tokens per chunk, one CTA per (request, head)) and returns once it has finished, so that
 * a device-side wait that ran out is returned as OLA_ERR_TIMEOUT (such calls from several host
 * threads run one at a time: they share one device error word per device); every other shape
 * runs token by token on CUDA cores and returns after the launch (stream-ordered).
 * Errors: INVALID_ARG, UNSUPPORTED, OOM, TIMEOUT, CUDA. */
ola_status ola_prefill(int32_t R, int32_t H, int32_t d_k, int32_t d_v, int32_t P,
                       int32_t in_dtype, const void* k, const void* v, const float* g,
                       const float* beta, float* S_out, void* stream);

/* ------------------------------------------------------------------ allocation-free decode
 * Not from the pages: the paper has no counterpart of this entry point. It serves callers that
 * may not allocate device memory while they decode: servers whose device memory is reserved up
 * front by an arena or caching allocator (a cudaMalloc behind its back can fail once the arena
 * holds the device, or fragment it), plugins loaded into a host application that owns every
 * device allocation, and latency-critical loops that cannot afford the device-wide
 * synchronisation a cudaMalloc / cudaFree can imply.
 *
 * ola_decode_noalloc runs a whole T_max-step decode of one GDN layer on the fp32 CUDA-core
 * replay path (same results as ola_create + T_max x ola_step + ola_destroy with
 * path = REPLAY, math = FP32), without creating a handle and without allocating anything:
 *   geom        : host pointer; path must be OLA_PATH_REPLAY and math OLA_MATH_FP32; T_max is
 *                 the number of steps decoded; the geometry limits are those of ola_create.
 *   S_ctx       : device [R][H][d_v][d_k] fp32 shared state (read only), 16-byte aligned.
 *   q, k        : device [T_max][R][B][H][d_k] in_dtype;  v : device [T_max][R][B][H][d_v]
 *                 (16-byte aligned).
 *   g, beta     : device [T_max][R][B][H] fp32;  parent_idx : device [T_max][R][B] int32
 *                 (4-byte aligned); parents as for ola_step, step by step.
 *   out_o       : device [T_max][R][B][H][d_v] fp32 (written), 16-byte aligned.
 * The transient state (transition records, ancestry rows, error word) lives in one fixed
 * device array of OLA_NOALLOC_SCRATCH_BYTES (16 MiB) inside the library, held by every GPU
 * that loads the library until the process exits. Problems needing more than that
 * (ola_noalloc_scratch_bytes) are rejected with OLA_ERR_SCRATCH_LIMIT, and bad geometry or
 * pointers with INVALID_ARG / UNSUPPORTED, before anything is queued. Every call shares the
 * array and leaves its contents behind (the call clears the error word itself); calls whose
 * work overlaps on the GPU (different streams, or several host threads) race on it and must be
 * serialised by the caller. The first call on each device resolves the array's device address
 * (a runtime query, no allocation); make that first call before any stream capture. The call
 * is synchronous: it waits for `stream` and returns the device error status (OLA_OK,
 * OLA_ERR_BAD_PARENT, ...) of this decode; on OLA_ERR_CUDA it has still waited for whatever
 * it had queued. */
#define OLA_NOALLOC_SCRATCH_BYTES (16u << 20)

uint64_t ola_noalloc_scratch_bytes(const ola_geometry* geom);

ola_status ola_decode_noalloc(const ola_geometry* geom, const float* S_ctx, const void* q,
                              const void* k, const void* v, const float* g, const float* beta,
                              const int32_t* parent_idx, float* out_o, void* stream);

/* ------------------------------------------------------ operators around the recurrence
 * Not from the pages: what a layer runs before and beside its recurrence. The pages take q, k
 * and v as given; a Gated DeltaNet layer makes them by a short causal convolution of its
 * projections and a norm of every query and key head (ola_conv, ola_conv_step, ola_qk_norm).
 * ola_scan and ola_scan_step are the recurrence of a selective state space layer: one scalar
 * decay per head and token, the same state [d_v][d_k], no erase term.
 *
 * Conventions, beside those above:
 * - Asynchronous on `stream`, no allocation, no host synchronisation: every call can be captured
 *   into a CUDA graph (the first call on each device looks up the library's error word: make it
 *   before a capture). Outputs must not overlap inputs unless a function says so.
 * - Strides are in elements, "tok" between consecutive tokens (or beams) and "seq" between
 *   sequences; 0 stands for the contiguous value. Channels (heads x width) are contiguous.
 *   A tok stride is at least the row's width; a sequence may not overlap the next one in outputs.
 *   No tensor may span more than 2^46 elements.
 * - lens: device [R] int32 or NULL: sequence r has min(max(lens[r], 0), P) tokens and the rows
 *   behind them are padding, never read into a result; the output rows there keep what they held.
 * - parent_idx: device [R][B] int32 or NULL: beam b continues state parent_idx[r][b] of the Bp
 *   states of its request. NULL: beam b continues state b (Bp = B) or the only one (Bp = 1). Out
 *   of range: clamped to 0 and OLA_ERR_BAD_PARENT is recorded. A state may have many children.
 * - Device-side errors (a bad parent, a bounded wait that ran out) go to one sticky word per
 *   device; the call carries on. ola_layer_status reads and clears it.
 * - Pointers to q, k, v, x, y, z and states: aligned to their element; 16-byte aligned pointers and
 *   rows (strides) run on wide accesses and TMA copies. fp32 pointers: 4 bytes.
 * - Forward only, like every operator of the library: nothing is kept for gradients. */

/* Wait for `stream`, return the first device-side error that a call of this section recorded on
 * the current device since the last ola_layer_status (OLA_OK if none), and clear it. There is one
 * word for all streams and threads: reading and clearing are one step, and an error goes to one of
 * several callers. Not to be called while `stream` is being captured. Errors: CUDA. */
ola_status ola_layer_status(void* stream);

/* Short depthwise causal convolution of W taps over u = state ++ x (the W-1 tokens before the
 * sequence, zeros if state_in is NULL):
 *   y[r][p][c] = act(bias[c] + sum_{i<W} w[c][i] u[r][p + i][c]),   act = identity or
 *   SiLU(u) = u / (1 + exp(-u));  sums in fp32, y rounded once to in_dtype.
 *   x         : [R][P][C] in_dtype (strides);  w : [C][W] fp32;  bias : [C] fp32 or NULL
 *   state_in  : [R][W-1][C] in_dtype, oldest token first, or NULL;  may be state_out itself
 *   y         : [R][P][C] in_dtype (strides);  y and x may be column slices of one wide buffer,
 *               but not the same columns
 *   state_out : [R][W-1][C] in_dtype or NULL: the last W-1 tokens of u up to the sequence's end
 * R >= 1, P 0..2^30 (P = 0: state_out = state_in), C >= 1, W 2..4.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
typedef struct {
  int32_t R, P, C, W;
  int32_t in_dtype;               /* OLA_F32 or OLA_BF16 */
  int32_t silu;                   /* 1: SiLU, 0: identity */
  int64_t x_tok, x_seq, y_tok, y_seq;
} ola_conv_desc;
ola_status ola_conv(const ola_conv_desc* d, const void* x, const float* w, const float* bias,
                    const void* state_in, const int32_t* lens, void* y, void* state_out,
                    void* stream);

/* ola_conv for one token of each of B = d->P beams per request:
 *   x, y [R][B][C];  state_in [R][Bp][W-1][C];  state_out [R][B][W-1][C] (required): the parent's
 *   window without its oldest token, then x. state_out may be state_in itself if parent_idx is
 *   NULL and Bp = B. The window of beam b after a step is thus the last W-1 tokens of its chain.
 * B >= 1, Bp >= 1. Errors as ola_conv. */
ola_status ola_conv_step(const ola_conv_desc* d, int32_t Bp, const void* x, const float* w,
                         const float* bias, const void* state_in, const int32_t* parent_idx,
                         void* y, void* state_out, void* stream);

/* Norm of every query and key head, then the position rotation, in one pass:
 *   n = x * rsqrt(m + eps) (* w[i]),   m = mean of x^2 over the head, or (l2) their sum
 *   pairs (a, b) of the first `rot` dims: (a cos - b sin, b cos + a sin) with the angle
 *   pos * inv_freq[i] taken in fp64, i the pair's index; pairs are (i, i + rot/2), or with
 *   `pair` (2i, 2i + 1). Norm and rotation in fp32, rounded once to in_dtype.
 *   q [N][Hq][d], k [N][Hk][d] in_dtype with N tokens (q_tok, k_tok: strides); q_out, k_out the
 *   same with strides qo_tok, ko_tok; q_out may be q itself (same stride), k_out may be k.
 *   wq, wk : [d] fp32 or NULL;  positions : [N] int32;  inv_freq : [rot/2] fp32 (both may be
 *   NULL if rot = 0)
 * N >= 0, Hq >= 0, Hk >= 0 (q, q_out may be NULL if Hq = 0; so k), d a multiple of 8 up to 512,
 * rot a multiple of 16 up to d, eps >= 0, pointers and strides 16-byte aligned (wq, wk, positions
 * and inv_freq 4). eps = 0 gives NaN for an all-zero head, as the formula does. A non-finite
 * value stays within its head. Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
typedef struct {
  int64_t N;
  int32_t Hq, Hk, d;
  int32_t in_dtype;
  int32_t l2;                     /* 1: sum of squares, 0: mean of squares */
  int32_t rot;                    /* rotated dims, 0 = none */
  int32_t pair;                   /* 1: pairs (2i, 2i + 1), 0: (i, i + rot/2) */
  float eps;
  int64_t q_tok, k_tok, qo_tok, ko_tok;
} ola_qk_desc;
ola_status ola_qk_norm(const ola_qk_desc* d, const void* q, const void* k, const float* wq,
                       const float* wk, const int32_t* positions, const float* inv_freq,
                       void* q_out, void* k_out, void* stream);

/* Selective state space scan of a prompt: for each sequence r and head h, with the key group
 * g = h / (H / G), from S = S_in (zeros if NULL), token by token
 *   dt = softplus(dt[r][p][h] + dt_bias[h])  (softplus = 0: dt as given, plus dt_bias)
 *   S <- exp(dt A[h]) S + dt v k^T,   o = S q + D[h] v,   y = o * SiLU(z)   (z, D if given)
 *   v, z, y : [R][P][H][d_v] in_dtype (strides);  k, q : [R][P][G][d_k] in_dtype (strides)
 *   dt      : [R][P][H] fp32;  A, D, dt_bias : [H] fp32, D and dt_bias may be NULL
 *   S_in    : [R][H][d_v][d_k] fp32 or NULL;  S_out : the same, or NULL; may be S_in itself
 *   ws      : device scratch of ola_scan_workspace_bytes(d) bytes, 16-byte aligned (NULL if 0).
 *             Calls that may overlap on the GPU need scratch of their own.
 * d_k, d_v in {16, 32, 64, 128, 256}, G divides H, R * H <= 2^24, P 0..2^30. dt * A is taken to
 * be <= 0 (a decay); growth is computed as the formula says as long as no product of the decays of
 * a call overflows. A NaN or infinity makes not finite what the formula makes so and no earlier token,
 * other row or column; where the formula gives an infinity, the result may be a NaN. States and sums
 * are fp32. bf16 prompts with 16-byte aligned rows and d_k <= 128 run in chunks of 128 tokens on
 * tensor cores: keys, queries and v enter exactly; the token-to-token weights and the copy of
 * the state that meets the queries are rounded to bf16 on the way to y (y itself is bf16), the
 * products that build the state are not (S_out is good to fp32). Everything else runs token by
 * token in fp32. Long prompts of few sequences are cut into pieces that run side by side and
 * are joined through `ws`. Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
typedef struct {
  int32_t R, P, H, G, d_k, d_v;
  int32_t in_dtype;
  int32_t softplus;
  int64_t v_tok, v_seq, k_tok, k_seq, q_tok, q_seq, z_tok, z_seq, y_tok, y_seq;
} ola_scan_desc;
ola_status ola_scan_workspace_bytes(const ola_scan_desc* d, uint64_t* out_bytes);
ola_status ola_scan(const ola_scan_desc* d, const void* v, const float* dt, const float* A,
                    const void* k, const void* q, const float* D, const float* dt_bias,
                    const void* z, const float* S_in, const int32_t* lens, void* y, float* S_out,
                    void* ws, uint64_t ws_bytes, void* stream);

/* ola_scan for one token of each of B = d->P beams per request: v, z, y [R][B][H][d_v],
 * k, q [R][B][G][d_k], dt [R][B][H], state_in [R][Bp][H][d_v][d_k] fp32, state_out
 * [R][B][H][d_v][d_k] fp32 (required; state_in itself if parent_idx is NULL and Bp = B).
 * States 16-byte aligned. Token by token in fp32. Every beam's state is materialised, as on the
 * FullState path of the decoder: its memory and traffic grow with B * H * d_v * d_k. Errors as
 * ola_scan. */
ola_status ola_scan_step(const ola_scan_desc* d, int32_t Bp, const void* v, const float* dt,
                         const float* A, const void* k, const void* q, const float* D,
                         const float* dt_bias, const void* z, const float* state_in,
                         const int32_t* parent_idx, void* y, float* state_out, void* stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* OLA_H_ */
