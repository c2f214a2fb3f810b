/*
 * deltalog.h -- C ABI of the DeltaLog decode library for B200 (sm_100a).
 *
 * DeltaLog ("DeltaLog: Deferred Materialization of Recurrent States for
 * Linear Attention Decoding", Abstract and AI Summary) keeps each head's
 * recurrent state as a dense base plus a bounded log of recent compact
 * updates.  A decode step reads base + log, appends one compact factor
 * instead of writing the whole state back, and a periodic merge folds the
 * log into the base.  The model observes the same dense state as eager
 * decoding (up to floating-point rounding order).
 *
 * Recurrences (state S is d_v x d_k per head, row = value index, contiguous
 * along the key index):
 *   GDN   S_t = a_t S_{t-1} (I - b_t k_t k_t^T) + b_t v_t k_t^T,  o_t = S_t q_t
 *   KDA   S_t = S_{t-1} Diag(a_t) (I - b_t k_t k_t^T) + b_t v_t k_t^T,  o_t = S_t q_t
 *   RWKV6 (stored as the transpose of its d_k x d_v matrix)
 *         S_t = S_{t-1} Diag(w_t) + v_t k_t^T,
 *         o_t = S_{t-1} r_t + (sum_c r_c u_c k_c) v_t
 *   GDN-2 S_t = S_{t-1} Diag(a_t) (I - (e_t o k_t) k_t^T) + (w_t o v_t) k_t^T,
 *         o_t = S_t q_t   (e_t: erase gate per key channel, w_t: write gate
 *         per value row; the log is KDA's, u_t = w_t o v_t - S' (e_t o k_t))
 * With gamma_t the decay accumulated since the base was last merged and
 * u_t = b_t (v_t - a_t S_{t-1} k_t) (GDN; KDA uses S_{t-1}(a_t o k_t)),
 *   S_t = S_b Diag(gamma_t) + sum_i u_i (k_i o gamma_t / gamma_i)^T,
 * so one log entry is (u_i, k_i, log gamma_i); RWKV6 stores u_i = v_i.
 *
 * Conventions for every call:
 *   - Returns DL_OK (0) or a negative DL_ERR_* code.  Arguments are checked
 *     on the host before anything is enqueued; a failed check enqueues
 *     nothing and changes no state.
 *   - Device pointers are plain CUDA device addresses owned by the caller.
 *     The library never allocates device memory and never frees caller
 *     memory; a dl_state borrows the three buffers sized by dl_state_bytes
 *     for its whole life.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Calls are asynchronous on it and never synchronize, except
 *     dl_state_reset and dl_device_error, which say so.
 *   - One dl_state is used from one host thread and one stream at a time.
 *   - Floating-point results equal eager decoding up to rounding order, not
 *     bitwise: the log and the merge sum in a different order.
 */
#ifndef DELTALOG_H
#define DELTALOG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Recurrence family (the DeltaLog page builds it for GDN, KDA and RWKV6), plus
 * GDN-2 (Gated DeltaNet-2 abstract: separate channel-wise erase and write
 * gates; KDA when both are the same scalar). */
enum dl_variant { DL_GDN = 0, DL_KDA = 1, DL_RWKV6 = 2, DL_GDN2 = 3 };

/* Element type of q (r), k and v as stored by the caller. */
enum dl_dtype { DL_F32 = 0, DL_BF16 = 1 };

/* Status codes. */
enum dl_status {
  DL_OK = 0,
  DL_ERR_ARG = -1,         /* null pointer, bad size, bad enum, bad mode   */
  DL_ERR_ALIGN = -2,       /* a pointer violates the alignment rule        */
  DL_ERR_LOG_FULL = -3,    /* a sequence's log holds L entries: merge first */
  DL_ERR_CUDA = -4,        /* a CUDA runtime call or launch failed          */
  DL_ERR_UNSUPPORTED = -5, /* valid but not built (head size, dtype)        */
  DL_ERR_DEVICE = -6       /* a kernel recorded an error (dl_device_error)  */
};

/* dl_merge modes. */
enum dl_merge_mode {
  DL_MERGE_FULL = 0, /* fold the logs of sequences whose log holds L entries */
  DL_MERGE_ALL = 1   /* fold every non-empty log                            */
};

/* dl_config.flags */
enum dl_flags {
  /* The step kernel merges in place: a head whose append would fill its
   * log writes the merged base instead and leaves an empty log, so the log
   * is never full and dl_merge(DL_MERGE_FULL) has nothing to do. */
  DL_FLAG_FUSED_MERGE = 1,
  /* Bit 2 is reserved (DL_ERR_ARG if set). */
  /* Kaczmarz step size (KLA, GDN and KDA only): the `beta` argument of a
   * step carries the gate eta_t and the kernels use
   * beta_t = eta_t / (|k_t|_2^2 + kla_eps) ("Kaczmarz Linear Attention"
   * abstract), so the write projects exactly whatever the key's norm.
   * With kla_eps = 0 a zero key gives an infinite beta_t, and the outputs
   * are NaN exactly as the formula's are: use kla_eps > 0 where keys may
   * vanish.  Not for RWKV6 or GDN-2 (DL_ERR_ARG). */
  DL_FLAG_KLA = 4,
  /* int8 base quantized once per window ("LeapQuant" abstract: the state
   * is quantized only at the end of a window of tokens, and outputs inside
   * the window use the fixed low-bit state plus high-precision buffered
   * updates; here the window is the stretch between two merges of a
   * sequence's log, and the log stays fp32).  The base holds int8 codes
   * and one fp32 scale per value row:
   *   amax_j = max_c |x_jc|,  inv_j = 127 / amax_j,
   *   code_jc = round-half-even(x_jc * inv_j),  scale_j = amax_j / 127,
   * each an fp32 operation rounded once (rows with amax_j < 2^-120 store
   * zero codes and scale 0); the base value is code_jc * scale_j.  Every
   * merge (DL_MERGE_FULL, DL_MERGE_ALL, the fused merge) folds the log in
   * fp32 and requantizes the rows it writes; dl_state_reset and
   * dl_state_load_seqs quantize the states they load. */
  DL_FLAG_BASE_Q8 = 8
};

/* Layer configuration.  d_k, d_v in {64, 128}; 1 <= L <= 64; B, H >= 1 and
 * B*H*d_v*d_k < 2^40.  `flags` is a bitwise OR of dl_flags.  `step_split`
 * is into how many work items (of d_v / step_split rows) the step kernel
 * cuts one head: 0 picks the library's default (2 for GDN at d_v = 128,
 * else 1), otherwise 1, 2 or 4 with
 * d_v / step_split >= 32 (a performance knob only: results do not depend
 * on it). */
typedef struct dl_config {
  int32_t variant;    /* enum dl_variant */
  int32_t B;          /* sequences in the batch */
  int32_t H;          /* heads per sequence */
  int32_t d_k;        /* key (and q / r) size per head */
  int32_t d_v;        /* value size per head */
  int32_t L;          /* log capacity: entries per head before a merge */
  int32_t in_dtype;   /* enum dl_dtype of q/r, k, v */
  int32_t flags;      /* enum dl_flags */
  int32_t step_split; /* 0 (default), 1, 2 or 4 */
  float kla_eps;      /* epsilon of the KLA step size (DL_FLAG_KLA), >= 0 */
} dl_config;

typedef struct dl_state dl_state;

/* Sizes in bytes of the three device buffers a state borrows:
 *   base: fp32 [B, H, d_v, d_k]                 the dense base S_b; with
 *         DL_FLAG_BASE_Q8 int8 codes [B, H, d_v, d_k] followed, at the
 *         next 256-B boundary, by the fp32 row scales [B, H, d_v]
 *   log : per head L entries of u (fp32 [d_v]; in_dtype for RWKV6),
 *         k (in_dtype [d_k]) and log-decay g (fp32, [1] for GDN, [d_k]
 *         otherwise), laid out as three arrays [B,H,L,.], each 256-B aligned
 *   meta: two int32 fill arrays [B, H] (read and written alternately by
 *         successive steps) and a device error word, each 256-B padded.
 * Any output pointer may be NULL.  Errors: DL_ERR_ARG, DL_ERR_UNSUPPORTED. */
int dl_state_bytes(const dl_config* cfg, size_t* base_bytes, size_t* log_bytes,
                   size_t* meta_bytes);

/* Creates a state over caller-owned device buffers of at least the sizes
 * above, each 256-byte aligned (else DL_ERR_ALIGN).  The contents are
 * undefined until dl_state_reset.  Enqueues nothing.  The handle (host
 * memory) is owned by the library until dl_state_destroy. */
int dl_state_create(const dl_config* cfg, void* base, void* log, void* meta,
                    dl_state** out);

/* Loads a dense state and starts every log.  S0: fp32 [B, H, d_v, d_k]
 * device buffer 16-B aligned, or NULL for a zero state (an int8 base
 * stores Q(S0), quantized row by row as described at DL_FLAG_BASE_Q8).  fill0: host int32
 * [B] with 0 <= fill0[b] < L, or NULL for zeros; sequence b starts with
 * fill0[b] log entries that change nothing (u = 0, k = 0, g = 0), so its
 * first merge comes after L - fill0[b] steps (ragged batches sit at
 * different merge phases).  Clears the device error word.  Synchronizes
 * `stream` before returning (it copies the fill counts from host memory). */
int dl_state_reset(dl_state* st, const float* S0, const int32_t* fill0, void* stream);

/* Loads dense states into some sequences and empties their logs, leaving
 * every other sequence untouched: the slot admission of continuous
 * batching (a finished sequence's slot takes a new one).  seqs: host int32
 * [n], distinct, each in [0, B).  S: fp32 [n, H, d_v, d_k] device buffer
 * (16-B aligned; entry i is the state of sequence seqs[i]) or NULL for zero
 * states.  The loaded sequences' fills become 0.  Asynchronous on `stream`.
 * Errors: DL_ERR_ARG (bad or repeated index, n < 0), DL_ERR_ALIGN. */
int dl_state_load_seqs(dl_state* st, int n, const int32_t* seqs, const float* S, void* stream);

/* One decode step for all B*H heads (one kernel launch).  Defines: the
 * DeltaLog page, Abstract -- a decode step reads the base and the log and
 * appends compact update factors instead of writing the full state back.
 *   q: q_t (r_t for RWKV6)  [B, H, d_k] in_dtype
 *   k: k_t                  [B, H, d_k] in_dtype
 *   v: v_t                  [B, H, d_v] in_dtype
 *   decay: fp32, GDN alpha_t [B, H]; KDA and GDN-2 alpha_t [B, H, d_k];
 *          RWKV6 w_t [B, H, d_k]; every value in (0, 1]
 *   beta: fp32 [B, H] for GDN/KDA; GDN-2: the erase gate e_t [B, H, d_k];
 *         ignored (may be NULL) for RWKV6
 *   bonus: fp32 [H, d_k] RWKV6 u; GDN-2: the write gate w_t [B, H, d_v];
 *          ignored (may be NULL) otherwise
 *   o: fp32 [B, H, d_v] output o_t
 * All pointers 16-byte aligned device addresses.  Without
 * DL_FLAG_FUSED_MERGE, returns DL_ERR_LOG_FULL (enqueuing nothing) when
 * some sequence's log already holds L entries: call dl_merge first.
 * The launch carries each sequence's current fill (from the host-side
 * mirror) by value, so a CUDA graph captured around this call would replay
 * the fills of the captured step: do not capture it. */
int dl_decode_step(dl_state* st, const void* q, const void* k, const void* v,
                   const float* decay, const float* beta, const float* bonus,
                   float* o, void* stream);

/* Folds logs into the base: S_b <- S_b Diag(gamma) + sum_i u_i (k_i o
 * gamma / gamma_i)^T, then empties those logs.  Defines: the DeltaLog page,
 * Abstract -- periodic merge steps fold the log back into the dense base.
 * mode DL_MERGE_FULL folds the sequences whose log holds L entries,
 * DL_MERGE_ALL every non-empty log.  Enqueues nothing when no sequence qualifies.  Like
 * dl_decode_step, the launch carries the qualifying sequences and their
 * fills by value (do not capture it in a CUDA graph). */
int dl_merge(dl_state* st, int mode, void* stream);

/* Writes the dense state S_t = base folded with the log to S_out (fp32
 * [B, H, d_v, d_k], 16-B aligned, must not alias the base) without changing
 * the state.  An int8 base is dequantized (code * scale) before the fold.
 * Defines: the DeltaLog page, Abstract -- the model observes the same dense
 * state as in eager decoding; this call produces that state on demand. */
int dl_materialize(const dl_state* st, float* S_out, void* stream);

/* Eager dense step, the comparison point: reads and writes the whole fp32
 * state S [B, H, d_v, d_k] (16-B aligned) in place, same recurrence and
 * arguments as dl_decode_step.  Defines: the DeltaLog page, Abstract --
 * eager decoding writes the full recurrent state back after every token.  cfg->L and every flag but DL_FLAG_KLA are
 * ignored (the state is always fp32). */
int dl_eager_step(const dl_config* cfg, float* S, const void* q, const void* k,
                  const void* v, const float* decay, const float* beta,
                  const float* bonus, float* o, void* stream);

/* Copies the host-side fill counts (entries per sequence, int32 [B]). */
int dl_state_fill(const dl_state* st, int32_t* fill_out);

/* Releases the handle (not the borrowed buffers).  NULL is accepted. */
int dl_state_destroy(dl_state* st);

/* ------------------------------------------------------------------------
 * Operators around the recurrent step: the short causal convolution that
 * feeds q, k and v, the selective state space recurrence (whose state has the
 * layout of every other recurrence here), and the residual RMS norm that turns
 * a layer's rows into the next projection's input.  They keep no state of
 * their own: every buffer is the caller's, and the conventions above hold
 * (checks on the host first, asynchronous on `stream`, no device memory
 * allocated, tensors on the current device).  The prompt forms take packed
 * sequences: starts is a host array of n + 1 non-decreasing int32 from 0 to
 * 2^31 - 1024 (beyond that DL_ERR_ARG, as for B of dl_conv_step), and sequence
 * s holds the rows starts[s] .. starts[s+1] - 1 (it may be empty); rows outside
 * [starts[0], starts[n]) are neither read nor written.  Lengths
 * travel by value with the launch, so a captured CUDA graph replays the
 * captured lengths; the single-token forms and dl_norm depend on nothing but
 * their buffers.  Row strides (ld*) count elements and may exceed the row, so
 * a row may be a range of columns of a wider one; an output must not share
 * elements with an input unless its comment says so.  Each call's result does
 * not depend on how the work is split, but for the rounding of sums. */

/* Element type of dl_norm's output, beside DL_F32 and DL_BF16. */
enum dl_out_dtype { DL_E4M3 = 2 /* 8 bits: 4 exponent, 3 mantissa, largest value 448 (e4m3) */ };

/* dl_conv_config.flags */
enum dl_conv_flags {
  DL_CONV_SILU = 1 /* y * sigmoid(y) on the way out: fp32 rows to 8 * 2^-24 of its value where
                      that is normal, bf16 rows rounded once (-0 where it is below 2^-119) */
};

/* Depthwise causal convolution of width W in {2, 3, 4} over C channels. */
typedef struct dl_conv_config {
  int32_t C;        /* channels, >= 1 */
  int32_t W;        /* taps */
  int32_t in_dtype; /* enum dl_dtype of x, y and the states */
  int32_t flags;    /* enum dl_conv_flags */
} dl_conv_config;

/* y[t, c] = act(bias[c] + sum_j w[c, j] x[t - W + 1 + j, c]) for packed
 * sequences; rows before a sequence's first token come from its state.
 *   x, y: in_dtype rows of C (strides ldx, ldy >= C); y must not be x
 *   w: fp32 [C, W] (the last tap meets the current token); bias: fp32 [C] or NULL
 *   h0: in_dtype [n, W-1, C], each sequence's last W - 1 input rows, oldest
 *       first, or NULL for zeros;  h1: the same after the call, or NULL;
 *       h1 may be h0.  An empty sequence passes its state on.
 * Pointers need their element's alignment only; pointers and strides of x, y
 * and the states in units of four elements, w and bias 16-byte aligned, and C a
 * multiple of 4 take the wide path.
 * Errors: DL_ERR_ARG, DL_ERR_ALIGN, DL_ERR_UNSUPPORTED (W). */
int dl_conv_prompt(const dl_conv_config* cfg, int32_t n, const int32_t* starts, const void* x,
                   int64_t ldx, const float* w, const float* bias, const void* h0, void* h1,
                   void* y, int64_t ldy, void* stream);

/* The same for one token of each of B sequences: row b of x and y, and the
 * state h [B, W-1, C], which is updated in place. */
int dl_conv_step(const dl_conv_config* cfg, int32_t B, const void* x, int64_t ldx, const float* w,
                 const float* bias, void* h, void* y, int64_t ldy, void* stream);

/* dl_ssm_config.flags */
enum dl_ssm_flags { DL_SSM_SOFTPLUS = 1 /* dt = softplus(dt_raw + dt_bias) */ };

/* Selective state space recurrence with a scalar decay per head and token:
 *   dt = dt_raw + dt_bias (through softplus with DL_SSM_SOFTPLUS), dt >= 0
 *   S_t = e^{dt a_h} S_{t-1} + dt v_t k_t^T,   o_t = S_t q_t + d_h v_t
 * with S fp32 [d_v, d_k] per head, and q, k shared by the H / G heads of a
 * group (head h reads group h / (H / G)).  d_k, d_v in {64, 128}. */
typedef struct dl_ssm_config {
  int32_t H;        /* heads */
  int32_t G;        /* groups of q and k; divides H */
  int32_t d_k;
  int32_t d_v;
  int32_t in_dtype; /* enum dl_dtype of q, k, v and o */
  int32_t flags;    /* enum dl_ssm_flags */
} dl_ssm_config;

/* Rows of one call.  q, k, v and o: 16-byte aligned, strides multiples of 16
 * bytes.  a <= 0 and dt >= 0 keep every factor in (0, 1].  A value that is
 * not finite makes the outputs of its own sequence (and head, or group)
 * undefined from its 128-token tile on, and no others. */
typedef struct dl_ssm_io {
  const void* q;        /* [T, G, d_k] */
  const void* k;        /* [T, G, d_k] */
  const void* v;        /* [T, H, d_v] */
  const float* dt;      /* [T, H] dt_raw */
  const float* a;       /* [H] */
  const float* d;       /* [H] or NULL (zeros) */
  const float* dt_bias; /* [H] or NULL (zeros) */
  void* o;              /* [T, H, d_v] */
  int64_t ldq, ldk, ldv, lddt, ldo; /* row strides in elements */
} dl_ssm_io;

/* Bytes of device workspace dl_ssm_prompt needs for these lengths on the
 * current device (may be 0). */
int dl_ssm_bytes(const dl_ssm_config* cfg, int32_t n, const int32_t* starts, size_t* bytes);

/* Packed prompts.  S0: fp32 [n, H, d_v, d_k] states before the first token,
 * or NULL for zeros; S1: the states after the last, or NULL; S1 may be S0 (a
 * prompt taken in pieces).  The state of a sequence can be loaded by
 * dl_state_load_seqs or stepped by dl_ssm_step.  workspace: 256-byte aligned,
 * of workspace_bytes >= dl_ssm_bytes (NULL when that is 0), written by the
 * call: calls that may run at the same time need one each.
 * Decays, weights and states are fp32, and S1 is right to fp32's rounding for
 * both row types.  fp32 rows: o too, its sums in the order of the tokens.  bf16
 * rows: what o sums, in fp32, are products of values rounded to bf16 first (each
 * token's weight q.k dt e^{..}, or the state that q reads, once per term: 2^-8 of
 * it at most), before o's own rounding: 0.0022 of o's norm in all, of which o's
 * rounding alone makes 0.0017.  dl_ssm_step rounds o only. */
int dl_ssm_prompt(const dl_ssm_config* cfg, int32_t n, const int32_t* starts, const dl_ssm_io* io,
                  const float* S0, float* S1, void* workspace, size_t workspace_bytes,
                  void* stream);

/* One token of each of B sequences: row b of the io buffers and the state
 * S [B, H, d_v, d_k] (16-byte aligned), updated in place. */
int dl_ssm_step(const dl_ssm_config* cfg, int32_t B, const dl_ssm_io* io, float* S, void* stream);

/* Root-mean-square norm of rows, after the addition of a residual:
 *   h = x + res,  n = h / sqrt(mean(h^2) + eps) * w,  all in fp32 (a sum of
 *   squares beyond its range makes n = 0).
 * out_dtype DL_F32 / DL_BF16: out = n, rounded once.  DL_E4M3: per block of
 * `block` channels (0: the whole row) scale = amax / 448 and code =
 * e4m3(n * (448 / amax)), round to nearest even; a block with amax < 2^-120
 * stores zero codes and scale 0. */
typedef struct dl_norm_config {
  int32_t D;         /* row length, 1 .. 16384 */
  int32_t in_dtype;  /* enum dl_dtype of x, res and res_out */
  int32_t out_dtype; /* enum dl_dtype or DL_E4M3 */
  int32_t block;     /* DL_E4M3: 128 or 0; else 0 */
  float eps;         /* >= 0 */
} dl_norm_config;

/*   x, res, res_out: in_dtype rows of D (strides ldx, ldr, ldro); res may be
 *   NULL (h = x); res_out takes h rounded to in_dtype, may be NULL, and may be
 *   x or res (the residual stream updated in place).
 *   w: fp32 [D];  out: rows of D of out_dtype (stride ldo)
 *   scales: fp32 [rows, ceil(D / 128)], or [rows] with block 0; NULL unless DL_E4M3.
 * Pointers need their element's alignment only, as for dl_conv_prompt.
 * Errors: DL_ERR_ARG, DL_ERR_ALIGN, DL_ERR_UNSUPPORTED (D). */
int dl_norm(const dl_norm_config* cfg, int64_t rows, const void* x, int64_t ldx, const void* res,
            int64_t ldr, const float* w, void* res_out, int64_t ldro, void* out, int64_t ldo,
            float* scales, void* stream);

/* Reads and optionally clears the device error word that kernels set when
 * a bounded wait gives up or a device-side check fails (code 0 = none;
 * *head = first failing head).  Synchronizes `stream`.
 *   - A state has its own word (in its meta buffer).  A nonzero code after a
 *     step or a merge means some head's work was skipped part-way (a step
 *     may already have advanced that head's fill, a merge may have folded
 *     only some rows): the state is invalid until dl_state_reset.
 *   - `st` NULL reads the one word per device that every dl_eager_step call,
 *     dl_ssm_prompt call and dl_selftest_wait_timeout share: the first error
 *     recorded wins, so with overlapping calls the head index (for
 *     dl_ssm_prompt the block that gave up; its outputs and states are then
 *     undefined) may belong to either, and the self-test clears the word
 *     (erasing what an earlier call recorded). */
int dl_device_error(dl_state* st, int32_t* code, int32_t* head, int clear, void* stream);

/* Exercises the kernels' failure path on the current device without a
 * fault: one warp waits, with the same bounded wait the kernels use, on a
 * shared-memory barrier nothing completes; after about one second it gives
 * up, records the timeout in the device error word the eager kernel uses
 * and returns.  *code receives the recorded code (1 = wait timed out),
 * read back and cleared.  Synchronizes `stream`. */
int dl_selftest_wait_timeout(int32_t* code, void* stream);

/* Total kernels this library has launched in this process. */
uint64_t dl_launch_count(void);

/* Static text for a status code. */
const char* dl_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* DELTALOG_H */
