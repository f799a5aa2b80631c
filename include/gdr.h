/*
 * gdr.h - C ABI of libgdr: the gated delta rule (forward and VJP) on
 * AMD Instinct MI355X (gfx950).
 *
 * What is computed.  The pages this library follows all turn on the gated
 * delta rule ("Adding VJP for gated delta net", ml-explore/mlx pull request
 * 4565; "Two-pass optimization for channelwise gated delta rule kernel",
 * pytorch/executorch pull request 21020; "perf(gated_delta_net): fold q/k
 * L2-norm into the gated_delta_rule kernel", NVIDIA/Megatron-LM pull request
 * 5396).  Per batch b and value head h, a state S (Dv x Dk) evolves per
 * token t as
 *     S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,
 *     o_t = S_t q_t,
 * the published gated delta rule (Yang, Kautz & Hatamizadeh, ICLR 2025).
 *   - alpha_t = exp(g_t).  g is a scalar per (b, t, h), or, with
 *     GDR_CHANNELWISE, one value per key channel (the ExecuTorch page's
 *     channelwise kernel): then the decay diag(alpha_t) is applied to the
 *     state before the prediction, S_{t-1} diag(alpha_t) (I - beta k k^T).
 *   - With GDR_USE_QK_L2NORM, q_t and k_t are replaced by
 *     x * (sum x^2 + 1e-6)^(-1/2) over the key dim inside the kernels (the
 *     Megatron-LM page, "What"/"Why"); without it they are used as given.
 *   - GQA: q and k have Hk heads; value head h reads k/q head h / (Hv/Hk).
 *   - No output scale is applied.
 *
 * Memory.  The state is stored as H = S^T with layout [B, Hv, Dk, Dv]
 * (Dv contiguous), always fp32.  All tensors are dense, row-major and
 * contiguous:
 *   q, k          [B, T, Hk, Dk]     io_dtype
 *   v, dout       [B, T, Hv, Dv]     io_dtype
 *   g             [B, T, Hv] (scalar gate) or [B, T, Hv, Dk] (channelwise), fp32
 *   beta          [B, T, Hv]         fp32
 *   h0, ht, dh0, dht  [B, Hv, Dk, Dv] fp32
 *   o, dv         [B, T, Hv, Dv]     out_dtype
 *   dq, dk        [B, T, Hk, Dk]     out_dtype
 *   dg            same shape as g, fp32;  dbeta [B, T, Hv] fp32
 *
 * Ownership and threading.  Every tensor pointer, including the workspace,
 * is a DEVICE pointer owned by the caller.  The library never allocates,
 * frees or synchronises: calls validate, then enqueue kernels on
 * `hip_stream` (a hipStream_t; NULL = the default stream) and return.  Calls
 * on different streams may run concurrently if their buffers are disjoint.
 *
 * Errors.  All arguments are checked before anything is launched; on any
 * error nothing is written and a status other than GDR_OK is returned.  A
 * failed kernel launch returns GDR_ERR_HIP and the HIP error text is kept in
 * a thread-local string read by gdr_last_hip_error().  No exception or abort
 * crosses this boundary.  NaN/Inf inputs propagate and never trap.
 *
 * Supported sizes.  Dk == Dv, with Dk in {16, 128}; Hv % Hk == 0; T >= 0
 * (T == 0: forward copies h0, or zeros, into ht; backward copies dht, or
 * zeros, into dh0).  Every pointer must be 16-byte aligned, the workspace
 * 256-byte aligned.  Results are bitwise reproducible from run to run
 * (fixed reduction orders, no floating-point atomics).
 */
#ifndef GDR_H_
#define GDR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDR_ABI_VERSION 4

typedef enum gdr_status {
  GDR_OK = 0,
  GDR_ERR_NULL_ARG = 1,            /* a required pointer is NULL            */
  GDR_ERR_BAD_SHAPE = 2,           /* negative/zero sizes, Hv % Hk != 0     */
  GDR_ERR_UNSUPPORTED = 3,         /* a valid problem this build cannot run */
  GDR_ERR_BAD_ALIGNMENT = 4,       /* pointer not 16 B (workspace 256 B)    */
  GDR_ERR_WORKSPACE_TOO_SMALL = 5, /* ws_bytes below the *_workspace size   */
  GDR_ERR_HIP = 6,                 /* a HIP launch or copy failed           */
  /* Never returned.  Widens the type's range to every non-negative int, so
   * any status value a caller passes back (gdr_status_str) is a value of
   * the type in C++ as in C. */
  GDR_STATUS_MAX_ENUM = 0x7fffffff
} gdr_status;

typedef enum gdr_dtype { GDR_F32 = 0, GDR_BF16 = 1 } gdr_dtype;

/* How the time axis is processed.  Both are HIP kernels.
 *   SEQUENTIAL: one token after another, fp32 state on chip (the decode
 *     kernel; the MLX page's "sequential" VJP).  Every shape is supported.
 *   CHUNKED: tokens grouped in chunks of chunk_size; the work inside a chunk
 *     runs as dense matrix-core products (the MLX page's "chunked" VJP).
 *     Scalar gate: bf16 io uses fp16 matrix-core operands with fp32
 *     accumulation (Dk = 128, chunk_size 32 or 64), every other shape fp32
 *     matrix-core operands.  Channelwise gate: bf16 io, Dk = 128,
 *     chunk_size 32 or 64 only (see below).
 *   AUTO: CHUNKED when supported and T is at least 12 (gdr_forward), 6
 *     (gdr_backward) or 10 (gdr_backward with GDR_CHANNELWISE) on the fp16
 *     matrix-core path, 64 on the fp32 one, else SEQUENTIAL: below those
 *     lengths the sequential kernels are the faster of the two on MI355X.
 *
 * Range of the fp16 chunked path.  Its matrix-core operands (normalised
 * q / k, v and dout rows, T = (I + A)^-1, the chunk states it keeps) are
 * fp16, whose finite range is +-65504; accumulation and the carried state
 * are fp32.  bf16 inputs convert to fp16 exactly inside that range.  A
 * v or dout element beyond it (or a T entry beyond it, possible only with
 * beta outside (0, 1)) overflows to +-Inf in its operand, and the outputs
 * that depend on it come out non-finite (Inf or NaN), never finite and
 * wrong.  Inputs of that size need the SEQUENTIAL algorithm or fp32 io. */
typedef enum gdr_algo {
  GDR_ALGO_AUTO = 0,
  GDR_ALGO_SEQUENTIAL = 1,
  GDR_ALGO_CHUNKED = 2
} gdr_algo;

/* GDR_FUSED_GATES: g and beta carry pre-activations a and b; the kernels
 * use g = -softplus(a) = -log(1 + e^a) (so alpha = 1 / (1 + e^a)) and
 * beta = sigmoid(b), and gdr_backward returns dg = dL/da and dbeta = dL/db.
 * This folds the caller's gate preparation into the kernels, in the spirit
 * of the Megatron-LM page's L2-norm fold ("What"/"Why"); the activations are
 * this library's choice (the pages name none).  Works with every algorithm
 * and with GDR_CHANNELWISE (then a has g's per-channel shape). */
/* GDR_SAVE_CHUNKS: keep the forward's per-chunk work for the VJP (what a
 * training step's autograd saves), on the chunked algorithm with bf16 io,
 * Dk = Dv = 128, chunk_size 32 or 64 and a scalar gate; elsewhere (the
 * SEQUENTIAL algorithm, also when AUTO picks it; fp32 io; Dk = 16; the
 * channelwise gate) both calls ignore the flag, and gdr_keeps_chunks tells
 * which case a problem is.  gdr_forward then needs gdr_backward_workspace(p) bytes
 * of workspace (gdr_forward_workspace reports that size) and leaves the
 * chunk images (normalised q/k, gates, T = (I + A)^-1, P) and every
 * chunk's entry state there; gdr_backward with the same problem, the same
 * inputs and that workspace, untouched in between, reads them instead of
 * recomputing them (it skips the prep and the chunk-state pass).  The
 * library cannot check that contract: a workspace not written by such a
 * forward gives wrong gradients (never an out-of-bounds access). */
enum { GDR_USE_QK_L2NORM = 1u, GDR_CHANNELWISE = 2u, GDR_FUSED_GATES = 4u, GDR_SAVE_CHUNKS = 8u };

typedef struct gdr_problem {
  int64_t B, T;       /* batch, tokens                                      */
  int32_t Hk, Hv;     /* k/q heads, v heads (Hv % Hk == 0)                  */
  int32_t Dk, Dv;     /* key and value head dims                            */
  int32_t io_dtype;   /* gdr_dtype of q, k, v, dout                         */
  int32_t out_dtype;  /* gdr_dtype of o, dq, dk, dv                         */
  uint32_t flags;     /* GDR_USE_QK_L2NORM | GDR_CHANNELWISE | GDR_FUSED_GATES
                         | GDR_SAVE_CHUNKS                                    */
  int32_t algo;       /* gdr_algo                                           */
  int32_t chunk_size; /* CHUNKED only: 16, 32 or 64; 0 means 64             */
} gdr_problem;
/* With GDR_CHANNELWISE, GDR_ALGO_CHUNKED is supported with bf16 io,
 * Dk = Dv = 128 and chunk_size 32 or 64 (else GDR_ERR_UNSUPPORTED); its VJP
 * forms each chunk's gradients from the chunk states the chunk chains store,
 * the per-channel decay carried inside the chunk-local sums (matrix cores
 * below the diagonal blocks, matrix cores or exact fp32 sums on them).
 * AUTO picks the chunked kernels there from the lengths given above. */

/* *keeps = 1 when GDR_SAVE_CHUNKS takes effect for problem *p (whether or
 * not the flag is set in p->flags), i.e. when gdr_forward with the flag
 * leaves its chunks in the workspace for gdr_backward; else 0, and both
 * calls ignore the flag.  Returns the validation status of the problem;
 * *keeps is written only on GDR_OK. */
gdr_status gdr_keeps_chunks(const gdr_problem* p, int* keeps);

/* Workspace bytes the call needs for problem *p (0 is possible).  Returns
 * the same validation status gdr_forward/gdr_backward would for the shape
 * part of the problem; *bytes is written only on GDR_OK. */
gdr_status gdr_forward_workspace(const gdr_problem* p, size_t* bytes);
gdr_status gdr_backward_workspace(const gdr_problem* p, size_t* bytes);

/* Forward pass.  h0 may be NULL (zero initial state).  ht may be NULL (final
 * state not wanted) and may alias h0 exactly (in-place decode: each kernel
 * reads its whole part of the state before writing it).  o must not alias
 * any input.  ws may be NULL when the workspace size is 0. */
gdr_status gdr_forward(const gdr_problem* p, const void* q, const void* k,
                       const void* v, const float* g, const float* beta,
                       const float* h0, void* o, float* ht, void* ws,
                       size_t ws_bytes, void* hip_stream);

/* VJP of gdr_forward for the loss <dout, o> + <dht, ht>.  Without
 * GDR_SAVE_CHUNKS the backward is stateless: it takes the forward's raw
 * inputs (q, k unnormalised when the flag is set) and recomputes what it
 * needs.  h0 and dht may be NULL (zeros); dh0 may be NULL (not wanted).
 * dq, dk, dv, dg, dbeta are required and must not alias inputs. */
gdr_status gdr_backward(const gdr_problem* p, const void* q, const void* k,
                        const void* v, const float* g, const float* beta,
                        const float* h0, const void* dout, const float* dht,
                        void* dq, void* dk, void* dv, float* dg, float* dbeta,
                        float* dh0, void* ws, size_t ws_bytes,
                        void* hip_stream);

/* Allocation-free forward, for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): gdr_forward with the workspace taken from a fixed scratch
 * array of GDR_NOALLOC_SCRATCH_BYTES (64 MiB) that the library keeps on
 * every GPU it runs on until the process ends.  The call allocates and
 * frees nothing; the caller still owns q .. ht.  Limits: problems whose
 * gdr_forward_workspace exceeds the scratch return
 * GDR_ERR_WORKSPACE_TOO_SMALL before anything is launched (the chunked path
 * needs about 1.1 MiB per 64 tokens of each sequence at Hk = 16, Hv = 32,
 * D = 128; the sequential path needs none); GDR_SAVE_CHUNKS returns
 * GDR_ERR_UNSUPPORTED.  All calls on one GPU share that GPU's scratch, so
 * calls that overlap on one GPU (concurrent streams, threads) race: order
 * them on one stream.  The stream must belong to the current device. */
#define GDR_NOALLOC_SCRATCH_BYTES (64u << 20)
gdr_status gdr_forward_noalloc(const gdr_problem* p, const void* q, const void* k,
                               const void* v, const float* g, const float* beta,
                               const float* h0, void* o, float* ht, void* hip_stream);

/* Ragged (packed) batches: p->B sequences of different lengths laid end to
 * end along the token axis, for prefill of a batch of prompts.  cu_seqlens
 * (device memory, int64, B + 1 entries, 8-byte aligned) holds the row
 * offsets: sequence b is token rows cu_seqlens[b] .. cu_seqlens[b+1] - 1 of
 * q, k [rows, Hk, Dk], v, o, dout, dv [rows, Hv, Dv], g [rows, Hv] or
 * [rows, Hv, Dk], beta [rows, Hv], dq, dk, dg, dbeta likewise; h0, ht, dht,
 * dh0 stay [B, Hv, Dk, Dv], one state per sequence.  p->T is an upper bound
 * on every length: workspace sizes (gdr_forward_workspace /
 * gdr_backward_workspace of the same p) hold ceil(T / C) chunks per
 * sequence.  The library reads the offsets only on the device, so it cannot
 * check them: it clamps each length to [0, T] (tokens past T are neither
 * read nor written) and reads and writes only the rows the offsets name,
 * which must lie inside the caller's buffers.  A sequence of length 0
 * passes its state through (ht = h0, dh0 = dht).  Each sequence gives
 * exactly what a separate call on it would (this is not a feature of the
 * pages: an interface variant for batches of unequal prompts).
 * Supported: GDR_ALGO_SEQUENTIAL (every shape, both passes) and
 * GDR_ALGO_CHUNKED on its fp16 path (bf16 io, Dk = Dv = 128, chunk_size 32
 * or 64; scalar or channelwise gate; GDR_SAVE_CHUNKS with a scalar gate).
 * The fp32 chunked path (fp32 io or Dk = 16) returns GDR_ERR_UNSUPPORTED;
 * AUTO picks as for gdr_forward / gdr_backward. */
gdr_status gdr_forward_varlen(const gdr_problem* p, const int64_t* cu_seqlens,
                              const void* q, const void* k, const void* v,
                              const float* g, const float* beta,
                              const float* h0, void* o, float* ht, void* ws,
                              size_t ws_bytes, void* hip_stream);
gdr_status gdr_backward_varlen(const gdr_problem* p, const int64_t* cu_seqlens,
                               const void* q, const void* k, const void* v,
                               const float* g, const float* beta,
                               const float* h0, const void* dout,
                               const float* dht, void* dq, void* dk, void* dv,
                               float* dg, float* dbeta, float* dh0, void* ws,
                               size_t ws_bytes, void* hip_stream);

/* ---------------------------------------------------------------------------
 * Linear attention with a decay for each head: the recurrence above without
 * its prediction term,
 *     S_t = alpha_t S_{t-1} + k_t v_t^T  (Dk x Dv),   o_t = S_t^T q_t,
 * alpha_t = exp(g_t), and its VJP.  The layer that stands beside gated delta
 * layers in a model: same heads (value head h reads k/q head h / (Hv/Hk)),
 * same fp32 state [B, Hv, Dk, Dv], same ragged batches, no output scale, q
 * and k used as given.
 *
 * g is [B, T, Hv], or [Hv] with GDR_LINEAR_HEAD_DECAY (one constant factor
 * per head; dg is then [Hv], summed over all tokens), or NULL (alpha = 1).
 * Any g, -Inf included (a finite state is dropped there), is allowed; growth past
 * the fp32 range gives Inf or NaN.  GDR_ALGO_CHUNKED (AUTO picks it for longer
 * sequences) splits a factor between two tokens of a chunk (64) where it crosses
 * 16 of them: growth of up to 2^48 over any run of a chunk's tokens keeps every
 * term; more can give Inf or NaN, or lose a term that decays in between.
 *
 * Dk and Dv are multiples of 16 up to 256, independent of each other; q_row,
 * k_row, v_row are the elements between one token's row and the next of q, k
 * and v (0: dense), so that the three may be column ranges of one projection:
 * at least H * D, in whole 16-byte units.  Rows of a batch follow each other
 * at the same distance.  All other tensors are dense, as above.  A row, with
 * its gap, holds at most 2^22 elements, Hv * Dk too; B and Hv are at most 65535,
 * B * Hv * (2 ceil(Dk/64) + ceil(Dv/64)) at most 2^22, B * T, and in the VJP
 * B * T * Hk, at most 2^31 - 1 (else GDR_ERR_UNSUPPORTED).
 *
 * Results: sums, the state and everything returned in fp32 (an fp32 o, dq,
 * dk, dv, and ht, dg, dh0 always) carry fp32 accuracy also from bf16 inputs,
 * relative to the sums of their terms' absolute values.  dg's terms are those of
 * dg_t = sum_{r >= t} (q_r . dq_r - k_r . dk_r) + <S_T, dS_T>, which cancel:
 * where a head decays strongly, dg_t is far smaller than they are, and its
 * rounding is not.  Where alpha_t is 0 in fp32, dg_t is 0.  bf16 outputs are
 * rounded once from sums whose matrix-core operands hold 16 bits or more (24 in
 * dq and dk where dg is wanted: asking for it can move one of their values to the
 * next bf16).  Every row past a sequence's end, and rows that no sequence covers,
 * are neither read nor written.  Inf and NaN inputs propagate; with
 * GDR_ALGO_CHUNKED an Inf may come out as NaN, and either may reach earlier tokens
 * of its chunk of 64.
 *
 * GDR_ALGO_SEQUENTIAL runs token by token (decoding, with ht == h0 allowed);
 * its sums do not depend on how a sequence is cut into calls.
 * GDR_ALGO_CHUNKED groups tokens for the matrix cores.  GDR_ALGO_AUTO picks by
 * T, and has a kernel of its own for one token.  All take every supported
 * problem. */
enum { GDR_LINEAR_HEAD_DECAY = 1u };

typedef struct gdr_linear_problem {
  int64_t B, T;                /* batch (sequences), tokens (bound on them)   */
  int32_t Hk, Hv;              /* k/q heads, v heads (Hv % Hk == 0)           */
  int32_t Dk, Dv;              /* key and value head dims                     */
  int32_t io_dtype;            /* gdr_dtype of q, k, v, dout                  */
  int32_t out_dtype;           /* gdr_dtype of o, dq, dk, dv                  */
  uint32_t flags;              /* GDR_LINEAR_HEAD_DECAY                       */
  int32_t algo;                /* gdr_algo                                    */
  int64_t q_row, k_row, v_row; /* elements between token rows; 0: dense       */
} gdr_linear_problem;

gdr_status gdr_linear_forward_workspace(const gdr_linear_problem* p, size_t* bytes);
gdr_status gdr_linear_backward_workspace(const gdr_linear_problem* p, size_t* bytes);

/* h0 may be NULL (zeros); ht may be NULL (not wanted) and may be h0.  o must
 * not alias an input. */
gdr_status gdr_linear_forward(const gdr_linear_problem* p, const void* q, const void* k, const void* v,
                              const float* g, const float* h0, void* o, float* ht, void* ws, size_t ws_bytes,
                              void* hip_stream);

/* VJP for the loss <dout, o> + <dht, ht>, from the forward's inputs alone.
 * h0 and dht may be NULL (zeros); dg and dh0 may be NULL (not wanted; without
 * dg less is computed; dg needs g).  dq and dk are summed over the value
 * heads that share a key head.  Outputs must not alias inputs. */
gdr_status gdr_linear_backward(const gdr_linear_problem* p, const void* q, const void* k, const void* v,
                               const float* g, const float* h0, const void* dout, const float* dht, void* dq,
                               void* dk, void* dv, float* dg, float* dh0, void* ws, size_t ws_bytes,
                               void* hip_stream);

/* Ragged batches: cu_seqlens as for gdr_forward_varlen. */
gdr_status gdr_linear_forward_varlen(const gdr_linear_problem* p, const int64_t* cu_seqlens, const void* q,
                                     const void* k, const void* v, const float* g, const float* h0, void* o,
                                     float* ht, void* ws, size_t ws_bytes, void* hip_stream);
gdr_status gdr_linear_backward_varlen(const gdr_linear_problem* p, const int64_t* cu_seqlens, const void* q,
                                      const void* k, const void* v, const float* g, const float* h0,
                                      const void* dout, const float* dht, void* dq, void* dk, void* dv, float* dg,
                                      float* dh0, void* ws, size_t ws_bytes, void* hip_stream);

/* The ragged VJP with its token rows counted.  gdr_linear_backward_workspace
 * of a ragged problem has to hold B * T tokens, the longest sequence's length
 * for each; given `rows`, the rows of q, k, v, dout and g (cu_seqlens[B] and
 * uncovered rows behind it included), it holds one entry for each of them
 * where that is less.  The limit on B * T * Hk then is one on rows * Hk.
 * Every offset lies in [0, rows]; rows = 0 is a batch of empty sequences. */
gdr_status gdr_linear_backward_varlen_workspace(const gdr_linear_problem* p, int64_t rows, size_t* bytes);
gdr_status gdr_linear_backward_varlen_rows(const gdr_linear_problem* p, int64_t rows, const int64_t* cu_seqlens,
                                           const void* q, const void* k, const void* v, const float* g,
                                           const float* h0, const void* dout, const float* dht, void* dq, void* dk,
                                           void* dv, float* dg, float* dh0, void* ws, size_t ws_bytes,
                                           void* hip_stream);

/* ---------------------------------------------------------------------------
 * Group norm of the heads' outputs, with an affine map and an activation:
 * what a layer does with o of either recurrence.  x is [rows, groups,
 * channels] (tokens, heads, Dv: channels last); per row and group
 *     n = (x - mean) (mean (x - mean)^2 + eps)^(-1/2),   u = weight n + bias,
 *     y = u silu(z)  (z given)  |  silu(u)  (GDR_NORM_SILU)  |  u,
 * where mean is subtracted only with GDR_NORM_CENTER (without it: the root
 * mean square).  A row's groups stand alone: a causal model shares no
 * statistics between tokens.  weight and bias are fp32 [groups, channels], or
 * [channels] for all groups with GDR_NORM_SHARED_WEIGHT, or NULL (ones,
 * zeros).  channels is a multiple of 8 up to 512; x_row and z_row are the
 * elements between rows of x and z (0: dense; in whole 16-byte units).  There are
 * at most 65535 groups and 2^40 rows, and a row, with its gap, holds at most 2^22
 * elements (else GDR_ERR_UNSUPPORTED).
 * All arithmetic is fp32, outputs are rounded once.  z together with
 * GDR_NORM_SILU is GDR_ERR_UNSUPPORTED.  Outputs must not alias inputs. */
enum { GDR_NORM_CENTER = 1u, GDR_NORM_SILU = 2u, GDR_NORM_SHARED_WEIGHT = 4u };

typedef struct gdr_norm_problem {
  int64_t rows;
  int32_t groups, channels;
  int32_t io_dtype;            /* gdr_dtype of x, z, dy                       */
  int32_t out_dtype;           /* gdr_dtype of y, dx, dz                      */
  uint32_t flags;              /* GDR_NORM_*                                  */
  float eps;                   /* >= 0                                        */
  int64_t x_row, z_row;        /* elements between rows; 0: dense             */
} gdr_norm_problem;

gdr_status gdr_group_norm_forward(const gdr_norm_problem* p, const void* x, const float* weight, const float* bias,
                                  const void* z, void* y, void* hip_stream);

/* VJP from the forward's inputs: dx [rows, groups, channels]; dz likewise
 * (required with z, ignored without); dweight, dbias in the parameters' shape,
 * fp32, either may be NULL (not wanted; with neither no workspace is needed),
 * and may be wanted where the parameter itself is NULL. */
gdr_status gdr_group_norm_backward_workspace(const gdr_norm_problem* p, size_t* bytes);
gdr_status gdr_group_norm_backward(const gdr_norm_problem* p, const void* x, const float* weight, const float* bias,
                                   const void* z, const void* dy, void* dx, void* dz, float* dweight, float* dbias,
                                   void* ws, size_t ws_bytes, void* hip_stream);

/* ---------------------------------------------------------------------------
 * The attention layer that stands beside the recurrent ones: rotary positions,
 * a paged cache of keys and values, attention of one new token over it, and
 * causal attention over whole sequences with its VJP.  Query head h reads
 * key/value head h / (Hq / Hk).  Head dims D are multiples of 16 up to 256 (the
 * same for keys and values), io is fp32 or bf16.  All sums, the softmax's
 * statistics and angles are held in fp32 or more; outputs are rounded once.
 *
 * Rotary positions.  Pair i < R / 2 of a head's first R channels, (i, i + R/2)
 * or with GDR_ROTARY_ADJACENT (2i, 2i + 1), is turned by the angle
 * pos[axis(i)] * freq[i]:
 *     (a, b) -> (a cos - b sin, b cos + a sin);   channels from R on stay.
 * The angle is formed and reduced in 64 bits, so far positions keep their
 * precision.  freq is fp32 [R / 2], pos int64 [axes, rows]: one position for
 * each axis (time, height, width).  section[a] pairs belong to axis a, summing
 * to R / 2: the first section[0] to axis 0, the next to axis 1 and so on; with
 * GDR_ROTARY_CYCLED pair i belongs to axis i % axes where i < axes *
 * section[i % axes], else to axis 0 (then axes * (section[a] - 1) + a < R / 2
 * for a > 0).  With one axis section is not read.  R is a multiple of 16. */
enum { GDR_ROTARY_ADJACENT = 1u, GDR_ROTARY_CYCLED = 2u };

typedef struct gdr_rotary {
  int32_t R;                   /* channels turned: 0 .. D                     */
  int32_t axes;                /* 1 .. 4                                      */
  int32_t section[4];          /* pairs of each axis                          */
  uint32_t flags;              /* GDR_ROTARY_*                                */
} gdr_rotary;

typedef struct gdr_rotary_problem {
  int64_t rows;                /* tokens                                      */
  int32_t Hq, Hk, D;           /* heads of q and of k (Hk 0: no k)            */
  int32_t io_dtype, out_dtype; /* gdr_dtype of q and k; of their outputs      */
  gdr_rotary rot;
  int64_t q_row, k_row;        /* elements between token rows; 0: dense       */
  int64_t qo_row, ko_row;      /* the same of the outputs                     */
} gdr_rotary_problem;

/* q [rows, Hq, D] and k [rows, Hk, D] turned into q_out and k_out.  An output
 * may be its own input (same dtype and row distance: in place) and must not
 * overlap an input otherwise.  backward is the VJP: the outputs' gradients in,
 * the inputs' out (the opposite turn); freq and pos have no gradients.  A row
 * holds at most 2^22 elements; rows lie at most 2^40 apart, in whole 16-byte
 * units; at most 2^31 - 1 rows. */
gdr_status gdr_rotary_forward(const gdr_rotary_problem* p, const void* q, const void* k, const int64_t* pos,
                              const float* freq, void* q_out, void* k_out, void* hip_stream);
gdr_status gdr_rotary_backward(const gdr_rotary_problem* p, const void* dq_out, const void* dk_out,
                               const int64_t* pos, const float* freq, void* dq, void* dk, void* hip_stream);

/* A paged cache.  Keys and values lie in two buffers of the same layout:
 * element (page, slot, head, channel) at page * page_stride + slot *
 * token_stride + head * head_stride + channel, no two of them in one place; all
 * strides 0 means dense [pages, page_size, Hk, D].  Strides are whole 16-byte
 * units, and a buffer spans less than 64 GiB.  table (device, int32, [B,
 * max_pages], rows table_row elements apart, 0: dense) holds each sequence's
 * pages in order: place j of a sequence is slot j % page_size of page
 * table[b][j / page_size].  An entry outside [0, pages) is a page that is not
 * there: nothing is stored to it, and its tokens are not visible (with pages 0 the
 * buffers may be NULL).  lengths (device, int64 [B]) are the tokens that each
 * sequence holds. */
typedef struct gdr_cache {
  int64_t pages;
  int32_t page_size, Hk, D;
  int32_t dtype;               /* gdr_dtype of keys and values                */
  int64_t page_stride, token_stride, head_stride;
  int32_t max_pages;
  int64_t table_row;
} gdr_cache;

/* Appending.  k and v [B, T, Hk, D] are the last T tokens of sequences that
 * hold lengths[b] tokens with them; token t gets place lengths[b] - T + t.  k
 * is turned (rot.R > 0) and stored in the cache's dtype, v is stored; with q
 * [B, T, Hq, D], the turned q is written to q_out (cache dtype).  pos [axes, B,
 * T] gives the positions; NULL: each token's place (one axis only).  A token
 * without a place (negative, or past the table) is not stored, its q is still
 * turned.  No two tokens of a call may have one slot (two sequences must not
 * append to one page): one of them, or a mixture, would remain.  varlen:
 * sequence b's new tokens are rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of
 * `rows` rows, its last ones; p->T bounds their number, tokens past it are not
 * stored; rows that no sequence covers are neither read nor written.  Row
 * distances as for gdr_rotary_forward; B is at most 65535, B * T and rows at most
 * 2^31 - 1. */
typedef struct gdr_append_problem {
  int64_t B, T;                /* sequences; new tokens of each (or a bound)  */
  int64_t rows;                /* varlen: rows of q, k, v                     */
  int32_t Hq;                  /* heads of q (0: no q)                        */
  int32_t io_dtype;            /* gdr_dtype of q, k, v                        */
  gdr_rotary rot;
  gdr_cache cache;
  int64_t q_row, k_row, v_row; /* elements between token rows; 0: dense       */
} gdr_append_problem;

gdr_status gdr_cache_append(const gdr_append_problem* p, const int64_t* lengths, const int32_t* table,
                            const void* q, const void* k, const void* v, const int64_t* pos, const float* freq,
                            void* q_out, void* k_cache, void* v_cache, void* hip_stream);
gdr_status gdr_cache_append_varlen(const gdr_append_problem* p, const int64_t* cu_seqlens, const int64_t* lengths,
                                   const int32_t* table, const void* q, const void* k, const void* v,
                                   const int64_t* pos, const float* freq, void* q_out, void* k_cache,
                                   void* v_cache, void* hip_stream);

/* Attention of one new token for each sequence over the cache, the token's own
 * key and value in it already:
 *     o = sum_j P_j v_j,  P = softmax_j(scale q . k_j)
 * over the places j < lengths[b] with window == 0, or lengths[b] - 1 - j <
 * window, or j < sinks.  q [B, Hq, D] in the cache's dtype (rows q_row
 * elements apart, 0: dense), o [B, Hq, D] in out_dtype, lse [B, Hq] fp32 the
 * logarithm of the softmax's sum (NULL: not wanted).  A sequence without a
 * visible token, or whose visible scores are all -Inf, gives o = 0 and lse =
 * -Inf.  What the pages hold in places that are not visible is never used; an Inf
 * in a visible v may come out as NaN.
 * Lengths are read on the device; they are clamped to [0, max_len], and max_len
 * (0: max_pages * page_size, which it may not exceed) sizes the workspace and
 * the launch, so a captured call serves all lengths up to it (at most 2^30).  B
 * and Hq are at most 65535, B * Hq at most 2^22, scale > 0, window and sinks >= 0.
 * Outputs must not alias inputs. */
typedef struct gdr_cache_attention_problem {
  int64_t B;
  int32_t Hq;
  int32_t out_dtype;
  gdr_cache cache;
  int64_t q_row;
  int64_t max_len;
  int64_t window, sinks;       /* window 0: all tokens                        */
  float scale;
} gdr_cache_attention_problem;

gdr_status gdr_cache_attention_workspace(const gdr_cache_attention_problem* p, size_t* bytes);
gdr_status gdr_cache_attention(const gdr_cache_attention_problem* p, const void* q, const void* k_cache,
                               const void* v_cache, const int32_t* table, const int64_t* lengths, void* o,
                               float* lse, void* ws, size_t ws_bytes, void* hip_stream);

/* Causal attention over whole sequences: token i sees token j of its sequence
 * where j <= i and (window == 0, or i - j < window, or j < sinks).  q, o, dout
 * [B, T, Hq, D], k, v [B, T, Hk, D], lse fp32 [B, T, Hq].  The VJP takes the
 * forward's inputs and its o and lse; dk and dv are summed over the query heads
 * that share a key head, in a fixed order.  bf16 outputs are rounded once: the
 * probabilities (and in the VJP their gradients) enter the matrix cores as two
 * bf16 operands, as three for fp32 outputs; fp32 io is fp32 throughout.  varlen:
 * cu_seqlens as for gdr_forward_varlen.  Outputs must not alias inputs.  NaN and
 * Inf propagate: scores that are
 * +Inf, or all -Inf, give NaN; an Inf in v or dout may come out as NaN, and Inf or
 * NaN in a token's v, k, q or dout may reach tokens of its sequence that are
 * masked from it but share a tile of 64 with ones that are not.  B and Hq are at
 * most 65535, T at most 2^22 - 128, a row, with its gap, at most 2^22 elements, B *
 * Hq * ceil(T / 128) at most 2^22, token rows at most 2^31 - 1 (else
 * GDR_ERR_UNSUPPORTED). */
typedef struct gdr_attention_problem {
  int64_t B, T;
  int32_t Hq, Hk, D;
  int32_t io_dtype;            /* gdr_dtype of q, k, v, dout                  */
  int32_t out_dtype;           /* gdr_dtype of o, dq, dk, dv                  */
  int64_t window, sinks;
  float scale;
  int64_t q_row, k_row, v_row; /* elements between token rows; 0: dense       */
} gdr_attention_problem;

gdr_status gdr_attention_forward(const gdr_attention_problem* p, const void* q, const void* k, const void* v, void* o,
                                 float* lse, void* hip_stream);
gdr_status gdr_attention_forward_varlen(const gdr_attention_problem* p, const int64_t* cu_seqlens, const void* q,
                                        const void* k, const void* v, void* o, float* lse, void* hip_stream);
/* `rows`: token rows of q (B * T, or a ragged batch's): they size the workspace, and
 * every offset lies in [0, rows]. */
gdr_status gdr_attention_backward_workspace(const gdr_attention_problem* p, int64_t rows, size_t* bytes);
gdr_status gdr_attention_backward(const gdr_attention_problem* p, const void* q, const void* k, const void* v,
                                  const void* o, const float* lse, const void* dout, void* dq, void* dk, void* dv,
                                  void* ws, size_t ws_bytes, void* hip_stream);
gdr_status gdr_attention_backward_varlen(const gdr_attention_problem* p, int64_t rows, const int64_t* cu_seqlens,
                                         const void* q, const void* k, const void* v, const void* o,
                                         const float* lse, const void* dout, void* dq, void* dk, void* dv, void* ws,
                                         size_t ws_bytes, void* hip_stream);

/* Per-kernel timing for benchmarks (not for use under graph capture).
 * While enabled, every kernel that gdr_forward / gdr_backward launch from the
 * calling thread is bracketed by a pair of HIP events recorded on the call's
 * stream (events are created on first use and recycled).  gdr_profile_read
 * waits for all recorded events, writes up to `cap` per-kernel entries
 * (static kernel name, summed milliseconds, launch count) to `out`, stores
 * the number of kernels seen in *n and clears the record.  Disabling drops
 * any unread record. */
typedef struct gdr_kernel_time {
  const char* name;
  double total_ms;
  int64_t launches;
} gdr_kernel_time;
gdr_status gdr_profile_enable(int on);
gdr_status gdr_profile_read(gdr_kernel_time* out, int cap, int* n);

const char* gdr_status_str(gdr_status s); /* static string, never NULL      */
const char* gdr_last_hip_error(void);     /* this thread's last HIP error   */
int gdr_abi_version(void);                /* GDR_ABI_VERSION                */

#ifdef __cplusplus
}
#endif

#endif /* GDR_H_ */
