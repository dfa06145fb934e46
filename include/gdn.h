/*
 * libgdn — chunked Gated DeltaNet on AMD Instinct MI355X (gfx950): the forward pass, its
 * backward pass, the decode operator with in-kernel gates and the causal conv1d before it; and
 * the operators of a selective state-space layer: the scan for prompts, its gradient and its
 * single-token form, the conv1d's gradient, and the group norm after a mixing layer; and those of a
 * linear attention block: the attention with a decay for each head for prompts, its gradient and its
 * single-token form, and the norms before and after a block with its gate and residual scale.
 *
 * The operation (one call): for every sequence n and value head h, with q/k head
 * hk = h / (H / Hg), starting from S = h0[n, h]^T (zero when h0 is NULL), for each token t
 *
 *     S   <- exp(g_t) S (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
 *     o_t <- scale S q_t
 *
 * and finally ht[n, h] = S^T.  It is evaluated chunk by chunk (chunk length C) through
 * the seven stages of the MegaGDN-PTO page (section 1.1: cumsum, transpose,
 * scaled_dot_kkt, solve_tril, wy_fast, chunk_h, chunk_o), either as seven launches
 * (GDN_VARIANT_STAGED) or as one launch that keeps every intermediate on chip
 * (GDN_VARIANT_FUSED; the megakernel idea of the page's section 1.3).  GQA (Hg q/k heads
 * shared by H value heads in contiguous groups) follows the page's section 5.2, packed
 * variable-length batches via cu_seqlens its section 5.3, and the user-level call shape
 * (q, k, v, g, beta, scale, initial_state, output_final_state) the FlashQLA how-to, step 5.2.
 *
 * Layouts (all contiguous, row-major; the token axis of a packed batch is B = 1, T = total):
 *   q, k    [B, T, Hg, Dk]   qkv_dtype (bf16 or f32)
 *   v, o    [B, T, H,  Dv]   qkv_dtype
 *   g       [B, T, H]        f32, the log-decay (g <= 0 in the intended use)
 *   beta    [B, T, H]        beta_dtype (bf16 or f32)
 *   h0, ht  [N, H, Dk, Dv]   f32 (the [B, H, K, V] state layout of the FlashQLA how-to,
 *                            step 5.3): ht[n, h, a, b] = S[b, a]
 *   cu_seqlens [N + 1]       int32, device memory, cu[0] = 0, non-decreasing, cu[N] <= B*T
 *
 * Ownership: the caller allocates and frees every buffer (device memory) and the optional
 * workspace.  The library keeps no pointer after a call returns, allocates nothing, and
 * has no mutable global state; calls are reentrant.  All work is enqueued on `stream`
 * (NULL = the default stream) and nothing is synchronised: errors found on the host are
 * returned before any launch; a launch failure returns GDN_ERR_HIP.  The buffers' device is the
 * calling thread's current one (work on its default stream goes there).  cu_seqlens is read
 * only on the device: values outside [0, B*T] are clamped (a sequence never reads or
 * writes outside the token range), but non-monotone values give unspecified results.
 *
 * Input domain: any finite bf16 (or f32) q, k, v and h0 go through every variant without
 * overflow of an intermediate (the fused kernel's matrix-core operands are bf16, with
 * fp32's exponent range).  The accuracy stated for bf16 (relative L2 5e-3 on o, 1e-2 on ht)
 * assumes the workloads' keys, L2-normalised with beta in [0, 1] (beta |k|^2 <= 2: the
 * fused kernel forms the 16 x 16 diagonal inverses in fp16, whose factors are then
 * bounded), and g <= 0.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gdn_status {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARG = 1, /* null required pointer, bad shape, misaligned pointer */
  GDN_ERR_UNSUPPORTED = 2, /* valid but not built: Dk != Dv, D not in {64,128,256}, ... */
  GDN_ERR_WORKSPACE = 3,   /* staged or segmented variant without the workspace it needs */
  GDN_ERR_HIP = 4          /* a HIP launch or attribute call failed */
} gdn_status;

typedef enum gdn_dtype { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype;

typedef enum gdn_variant {
  GDN_VARIANT_AUTO = 0,      /* recurrent for a few tokens per sequence (dense: T <= 8;
                                packed: B*T <= 8 N); else fused when built for the shape,
                                otherwise staged; segmented for a batch of few long
                                sequences (dense or packed) when the workspace for it is
                                given (fused otherwise)                                    */
  GDN_VARIANT_STAGED = 1,    /* seven launches, intermediates in the workspace */
  GDN_VARIANT_FUSED = 2,     /* one launch, one workgroup per (sequence, head) */
  GDN_VARIANT_SEGMENTED = 3, /* every sequence split into segments that run in parallel
                                (dense: S per sequence; packed: ceil(len / Ls) per sequence,
                                the table built on the device).  The state recurrence is
                                affine in the initial state, h_end = M h_in + b; the fused
                                kernel finds M (from h_in = I, v = 0) and b (from h_in = 0)
                                of every segment, a scan composes h_in(s+1) = M_s h_in(s) +
                                b_s (fp32), and a last fused pass writes o.  Three passes over
                                the data, many-fold parallelism (the long-prompt case of the
                                FlashQLA how-to, section 8.3).  Needs the workspace reported
                                for it.                                                    */
  GDN_VARIANT_RECURRENT = 4  /* token by token, the state kept in registers: one read and one
                                write of each (sequence, head) state per call, whatever the
                                number of tokens, and one dependent step per token.  For
                                decode (one or a few tokens per sequence; the per-token
                                delta-rule kernel of the TileLang × xLLM page).  Any dtype
                                and D the header lists; no workspace; chunk is ignored.
                                ht may be the same buffer as h0 (state updated in place).
                                The gates arrive as g and beta, as in every variant.       */
} gdn_variant;

/* Intermediate buffers of the staged variant, readable through gdn_stage_buffer().  The
 * fused variant's stage stop (stop_after = 6 with GDN_VARIANT_FUSED) writes the chunk
 * table, the sequences' first chunks, h_c and v_new only, at its own 64-token chunk. */
typedef enum gdn_buffer {
  GDN_BUF_CHUNK_TABLE = 0, /* int32 [max_chunks, 4]: (sequence, first token, length, index
                              in sequence); unused rows have length 0                  */
  GDN_BUF_SEQ_CHUNKS = 1,  /* int32 [N + 1]: first chunk of each sequence; [N] = total    */
  GDN_BUF_G_CUM = 2,       /* f32 [B*T, H]: in-chunk inclusive prefix sum of g  (stage 1) */
  GDN_BUF_G_T = 3,         /* f32 [H, B*T]: g_cum transposed                    (stage 2) */
  GDN_BUF_BETA_T = 4,      /* beta_dtype [H, B*T]: beta transposed              (stage 2) */
  GDN_BUF_A = 5,           /* f32 [B*T, H, C]: gated strictly-lower K K^T       (stage 3) */
  GDN_BUF_TINV = 6,        /* qkv_dtype [B*T, H, C]: rows of (I + A)^-1         (stage 4) */
  GDN_BUF_W = 7,           /* qkv_dtype [B*T, H, Dk]                            (stage 5) */
  GDN_BUF_U = 8,           /* qkv_dtype [B*T, H, Dv]                            (stage 5) */
  GDN_BUF_H_C = 9,         /* qkv_dtype [max_chunks, H, Dk, Dv]: state at chunk start (6) */
  GDN_BUF_V_NEW = 10,      /* qkv_dtype [B*T, H, Dv]: U - W h_c                 (stage 6) */
  GDN_BUF_COUNT = 11
} gdn_buffer;

typedef struct gdn_desc {
  int32_t B, T;       /* dense batch [B, T, ...]; packed varlen: B = 1, T = total tokens */
  int32_t N;          /* sequences: B when cu_seqlens is NULL, else len(cu_seqlens) - 1 */
  int32_t H, Hg;      /* value heads, q/k heads; H % Hg == 0                              */
  int32_t Dk, Dv;     /* head dims; this build supports Dk == Dv in {64, 128, 256}        */
  int32_t chunk;      /* C in {64, 128} (0 selects 128): the chunk length of the staged
                         variant.  The fused and segmented variants run their own chunk
                         (64 tokens, 32 at D = 256: what three K/Q buffers allow in LDS) and
                         the recurrent one goes token by token, whatever C asks for; the
                         result is the same up to rounding (the chunked form is exact for
                         any chunk length).  gdn_resolved_chunk() reports the length run.  */
  int32_t qkv_dtype;  /* gdn_dtype of q, k, v, o                                          */
  int32_t beta_dtype; /* gdn_dtype of beta                                                */
  int32_t variant;    /* gdn_variant                                                      */
  int32_t stop_after; /* 0 = the whole pass.  Staged: k in 1..6 stops after stage k (the
                         page's section 7.4 debugging mode).  Fused: 6 only, and only for
                         bf16 with D in {64, 128}: the kernel keeps every stage on chip and
                         forms just the chunk-start states and v_new, which it then writes
                         to the workspace (GDN_BUF_H_C, GDN_BUF_V_NEW, at 64-token chunks)
                         instead of o; it never forms G, A, T, W or U, so 1..5 are refused
                         (GDN_ERR_UNSUPPORTED), as is any stop for the other variants.    */
  void* workspace;    /* device memory for the staged and segmented variants and the fused
                         variant's longest-first order (256-byte aligned; may be NULL for
                         fused, see gdn_chunk_fwd_workspace_size)                         */
  size_t workspace_bytes;
  int32_t grad_dtype; /* gdn_chunk_bwd only: gdn_dtype of dq, dk, dv.  GDN_F32 (0, the
                         default) or, with bf16 inputs, GDN_BF16 (the gradients rounded
                         once, at the store; half the bytes written).  Ignored by the
                         forward entry points.                                            */
} gdn_desc;

/* Causal depthwise 1-D convolution with a decode state: the step before the gated delta
 * rule (the causal_conv1d operator of the TileLang × xLLM page).  For sequence n, channel
 * c and position t of the sequence, with x~ = (the W - 1 inputs before the sequence, taken
 * from the sequence's state line, or zeros) followed by the sequence's inputs,
 *
 *     y[t, c] = act(bias[c] + sum_{i < W} weight[c, i] x~[t + i, c])
 *
 * (weight[c, W - 1] multiplies the current token) and, when conv_state is given, the line
 * afterwards holds the last W - 1 entries of x~ (part of the old line when the sequence is
 * shorter than W - 1).  act is the identity or SiLU (z sigmoid(z)), in fp32.
 *
 * Layouts (contiguous, row-major; channels contiguous so that a token's row is one read):
 *   x, y        [B, T, C]            dtype (bf16 or f32); packed: B = 1, T = total tokens
 *   weight      [C, W]               f32
 *   bias        [C]                  f32, or NULL (zero)
 *   conv_state  [state_lines, W - 1, C]  dtype, or NULL (zeros in, nothing written); read
 *                                    and written in place
 *   cache_indices      [N] int32 or NULL (sequence n uses line n): an index outside
 *                      [0, state_lines) gives a zero start and leaves every line untouched
 *   has_initial_state  [N] int32 or NULL (all start from their line): 0 = start from zeros
 *   cu_seqlens         [N + 1] int32 or NULL (dense batch), as for gdn_chunk_fwd
 * C is a multiple of 8 and W is 2, 3 or 4; pointers are device pointers, x, y and conv_state
 * 16-byte aligned; weight is required, x and y too unless B*T = 0.  Two sequences naming the same line give unspecified lines.  Errors are
 * returned before any launch; the work is enqueued on `stream` (two launches: outputs, then
 * the state lines). */
typedef enum gdn_activation { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1 } gdn_activation;

typedef struct gdn_conv_desc {
  int32_t B, T;        /* dense [B, T, C]; packed: B = 1, T = total tokens              */
  int32_t N;           /* sequences: B (or 0) for a dense batch, len(cu_seqlens) - 1     */
  int32_t channels;    /* C                                                             */
  int32_t width;       /* W                                                             */
  int32_t dtype;       /* gdn_dtype of x, y and conv_state                              */
  int32_t activation;  /* gdn_activation                                                */
  int32_t state_lines; /* lines in conv_state                                           */
} gdn_conv_desc;

gdn_status gdn_causal_conv1d_fwd(const gdn_conv_desc* d, const void* x, const float* weight,
                                 const float* bias, void* conv_state,
                                 const int32_t* cache_indices,
                                 const int32_t* has_initial_state, const int32_t* cu_seqlens,
                                 void* y, hipStream_t stream);

/* The selective state-space scan, a linear recurrence with a diagonal state next to the delta
 * rule's matrix state.  For every sequence n, channel c (of group g = c / (channels / groups))
 * and state s < dstate, from h = h0[n, c, :] (zero when h0 is NULL), for each token t
 *
 *     step  = softplus(dt[t, c] + dt_bias[c])        (dt[t, c] + dt_bias[c] without dt_softplus)
 *     h[s] <- exp(step A[c, s]) h[s] + step x[t, c] B[t, g, s]
 *     y[t, c] = (sum_s C[t, g, s] h[s] + D[c] x[t, c]) z sigmoid(z),   z = z[t, c]
 *
 * and finally ht[n, c, :] = h.  D NULL is zero, dt_bias NULL is zero, z NULL leaves the gate
 * out.  Decays, states and sums are fp32 whatever the dtype; y is rounded once.
 *
 * Layouts (row-major; a token's row is contiguous, the rows *_stride elements apart, over the
 * whole [B, T] token axis; 0 = rows one after another):
 *   x, dt, z   [B, T, channels]         dtype (bf16 or f32)
 *   Bm, Cm     [B, T, groups, dstate]   dtype
 *   y          [B, T, channels]         dtype, contiguous
 *   A          [channels, dstate]       f32 (negative in the intended use)
 *   D, dt_bias [channels]               f32
 *   h0, ht     [N, channels, dstate]    f32; cu_seqlens [N + 1] int32 as for gdn_chunk_fwd
 * Any channels, groups dividing it, dstate 1 .. 256.  GDN_ERR_UNSUPPORTED beyond 2^30 tokens,
 * 65536 sequences, 2^20 channels, launches of 2^32 threads, or where the rows of a sequence (of all
 * tokens of a packed batch) and one more, or of 257 tokens if it is longer, pass 2 GiB.  Pointers are
 * device pointers aligned to their element; errors are returned before any launch; nothing is
 * synchronised or allocated.
 * x, dt, A, Bm, Cm, y are required unless B*T = 0 (A always).  h0 and ht may be the same buffer.  y
 * of tokens of a packed batch that no sequence has is not written.  Few or long sequences are split
 * into chunks that run in parallel, so results depend on the descriptor in their last bits, never on
 * scheduling.  An infinity or a NaN in x, dt, z or dy reaches its own channel of its own sequence and
 * the gradients that sum over it (dB and dC of its group, the parameters'); what an infinity makes
 * there is not finite, but may be NaN where the formula has an infinity. */
typedef struct gdn_scan_desc {
  int32_t B, T;         /* dense [B, T, ...]; packed: B = 1, T = total tokens               */
  int32_t N;            /* sequences: B (or 0) for a dense batch, len(cu_seqlens) - 1       */
  int32_t channels;
  int32_t groups;       /* groups of channels that share B and C                            */
  int32_t dstate;       /* states a channel                                                 */
  int32_t dtype;        /* gdn_dtype of x, dt, z, Bm, Cm, y (and of their gradients)        */
  int32_t dt_softplus;  /* 0 or 1                                                           */
  int32_t state_lines;  /* gdn_selective_state_update only: lines of the pool               */
  int64_t x_stride, dt_stride, z_stride, b_stride, c_stride;
  void* workspace;      /* 256-byte aligned, as many bytes as the call's query gives        */
  size_t workspace_bytes;
} gdn_scan_desc;

/* Bytes of workspace gdn_selective_scan_fwd needs (dense and packed alike: N other than 0 or B
 * is a packed batch; B == 1 may be either).  Host-only.  0 and *status set when refused. */
size_t gdn_selective_scan_workspace_size(const gdn_scan_desc* d, gdn_status* status);

gdn_status gdn_selective_scan_fwd(const gdn_scan_desc* d, const void* x, const void* dt,
                                  const float* A, const void* Bm, const void* Cm,
                                  const float* D, const void* z, const float* dt_bias,
                                  const float* h0, const int32_t* cu_seqlens, void* y, float* ht,
                                  hipStream_t stream);

/* Bytes of workspace gdn_selective_scan_bwd needs.  Host-only. */
size_t gdn_selective_scan_bwd_workspace_size(const gdn_scan_desc* d, gdn_status* status);

/* The gradient of gdn_selective_scan_fwd: the exact derivative of the recurrence, from the
 * forward's inputs (nothing of a forward call is kept) and the gradients of its outputs.
 *   dy                 [B, T, channels] dtype, contiguous
 *   dht                [N, channels, dstate] f32, or NULL (zero)
 *   dx, ddt, dz        [B, T, channels] dtype, contiguous (dz required with z)
 *   dB, dC             [B, T, groups, dstate] dtype, contiguous: summed over the channels that
 *                      share them in fp32, rounded once
 *   dA [channels, dstate], dD, ddt_bias [channels], dh0 [N, channels, dstate]  f32; dD, ddt_bias
 *                      and dh0 may be NULL (not written)
 * Sums are made in a fixed order (no atomics): the same call gives the same bits.  Gradients of
 * tokens of a packed batch that no sequence has are unspecified.
 * The workspace is larger than the inputs: beside B and C as fp32 rows it holds dB's and dC's partial
 * sums for every block of 64 channels of a group, 8 * B*T * dstate bytes a block (dstate rounded up
 * to 4, 8, 16 or a multiple of 32), and three sets of states for every chunk of 64 tokens (fewer in
 * small batches), 12 * channels * dstate bytes a chunk: 350 MB for 8 x 2048 tokens of 4096 channels
 * and 16 states, 1.36 GB with 64 states, 5.4 GB with 256. */
gdn_status gdn_selective_scan_bwd(const gdn_scan_desc* d, const void* x, const void* dt,
                                  const float* A, const void* Bm, const void* Cm,
                                  const float* D, const void* z, const float* dt_bias,
                                  const float* h0, const int32_t* cu_seqlens, const void* dy,
                                  const float* dht, void* dx, void* ddt, float* dA, void* dB,
                                  void* dC, float* dD, void* dz, float* ddt_bias, float* dh0,
                                  hipStream_t stream);

/* The same recurrence for one token of each of d->B sequences (T is 1, N is 0 or B), the states
 * in a pool: sequence b reads line cache_indices[b] (b when NULL) of state [state_lines,
 * channels, dstate] and writes line out_indices[b] (the line it read when NULL).  A line read
 * from outside the pool is a zero start, one written outside it is dropped.  A line that one
 * sequence writes and another reads or writes in the same call has unspecified contents.  Rows may
 * be any number of bytes apart.  No workspace. */
gdn_status gdn_selective_state_update(const gdn_scan_desc* d, float* state, const void* x,
                                      const void* dt, const float* A, const void* Bm,
                                      const void* Cm, const float* D, const void* z,
                                      const float* dt_bias, const int32_t* cache_indices,
                                      const int32_t* out_indices, void* y, hipStream_t stream);

/* The gradient of gdn_causal_conv1d_fwd.  With x~ each sequence's inputs behind the W - 1 before
 * it (initial [N, W - 1, C] dtype: its state line as it was before the forward, or NULL: zeros),
 * given dy and dfinal, the gradient of the state line afterwards ([N, W - 1, C] dtype, or NULL:
 * zero), it writes
 *   dx       [B, T, C]      dtype
 *   dweight  [C, W], dbias [C]   f32 sums over all tokens (NULL: not written)
 *   dinitial [N, W - 1, C]  dtype, the gradient of initial (NULL: not written)
 * d->state_lines is ignored; shapes, checks and the rest as for the forward (x, dy, dx, initial,
 * dfinal and dinitial 16-byte aligned; at most 65535 * 1024 channels).  Sums are made in a fixed
 * order.  dx of tokens of a packed batch that no sequence has is not written.  The workspace
 * (256-byte aligned, gdn_causal_conv1d_bwd_workspace_size bytes) is required when B*T > 0. */
size_t gdn_causal_conv1d_bwd_workspace_size(const gdn_conv_desc* d, gdn_status* status);

gdn_status gdn_causal_conv1d_bwd(const gdn_conv_desc* d, const void* x, const float* weight,
                                 const float* bias, const void* initial,
                                 const int32_t* cu_seqlens, const void* dy, const void* dfinal,
                                 void* dx, float* dweight, float* dbias, void* dinitial,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Linear attention with a decay for each head, the delta rule's recurrence without its correction.
 * For every sequence n and value head h with q/k head hk = h / (H / Hg), from S = h0[n, h] (zero when
 * h0 is NULL), for each token t
 *
 *     S   <- exp(g) S + k_t v_t^T          (k_t, q_t of head hk, v_t of head h)
 *     o_t <- scale S^T q_t
 *
 * and finally ht[n, h] = S.  g is a log-decay for each head (head_decay = 1) or each token and head.
 *
 * Layouts (row-major; a token's row is contiguous, the rows *_stride elements apart over the whole
 * [B, T] token axis; 0 = rows one after another):
 *   q, k    [B, T, Hg, Dk]   dtype (bf16 or f32)
 *   v, o    [B, T, H, Dv]    dtype; o contiguous
 *   g       [H] or [B, T, H] f32 (at most 0 in the intended use; -inf forgets the state)
 *   h0, ht  [N, H, Dk, Dv]   f32; cu_seqlens [N + 1] int32 as for gdn_chunk_fwd
 * Dk and Dv are multiples of 8 up to 256, equal or not; any H, Hg dividing it.  Pointers are device
 * pointers aligned to 16 bytes (g, cu_seqlens, indices: 4) and rows a multiple of 16 bytes apart.
 * GDN_ERR_UNSUPPORTED beyond 2^30 tokens, 65536 sequences, rows of 2^23 elements or launches of 2^32
 * threads.  Errors are returned before any launch; nothing is synchronised or allocated.
 * q, k, v, g, o are required unless B*T = 0.  h0 and ht may be the same buffer; no other output may
 * overlap an input.  o of tokens of a packed batch that no sequence has is not written.
 * States and sums are fp32.  In bf16, o is as near as fp32 sums rounded once (scores and the state that
 * meets q keep 16 bits or more on their way to it), ht as exact as fp32 sums.  Few or long sequences are
 * split into segments that run in parallel, so results depend on the descriptor in their last bits, never
 * on scheduling.
 * An infinity or a NaN in q, k, v or g reaches its own head (its q/k head's value heads) of its own
 * sequence, from the chunk it is in: the outputs of that chunk's earlier tokens may be NaN too.  One in h0
 * reaches its own head of its own sequence.  In bf16 an infinity in v or in a state may come out as a NaN. */
typedef struct gdn_linear_desc {
  int32_t B, T;         /* dense [B, T, ...]; packed: B = 1, T = total tokens               */
  int32_t N;            /* sequences: B (or 0) for a dense batch, len(cu_seqlens) - 1       */
  int32_t H, Hg;        /* value heads, q/k heads; H % Hg == 0                              */
  int32_t Dk, Dv;       /* head sizes                                                       */
  int32_t dtype;        /* gdn_dtype of q, k, v, o (and of dout, dq, dk, dv)                */
  int32_t head_decay;   /* 1: g [H]; 0: g [B, T, H]                                         */
  int32_t state_lines;  /* gdn_linear_state_update only: lines of the pool                  */
  float scale;          /* Dk^-0.5 is the usual choice                                      */
  int64_t q_stride, k_stride, v_stride;
  void* workspace;      /* 256-byte aligned, as many bytes as the call's query gives        */
  size_t workspace_bytes;
} gdn_linear_desc;

/* Bytes of workspace gdn_linear_attn_fwd needs: 0 where sequences stay whole (dense and packed
 * alike: N other than 0 or B is a packed batch; B == 1 may be either).  Host-only.  0 and *status set
 * when refused. */
size_t gdn_linear_attn_workspace_size(const gdn_linear_desc* d, gdn_status* status);

gdn_status gdn_linear_attn_fwd(const gdn_linear_desc* d, const void* q, const void* k,
                               const void* v, const float* g, const float* h0,
                               const int32_t* cu_seqlens, void* o, float* ht, hipStream_t stream);

/* Bytes of workspace gdn_linear_attn_bwd needs.  Host-only. */
size_t gdn_linear_attn_bwd_workspace_size(const gdn_linear_desc* d, gdn_status* status);

/* The gradient of gdn_linear_attn_fwd, from the forward's inputs (nothing of a forward call is kept)
 * and the gradients of its outputs.
 *   dout    [B, T, H, Dv]  dtype, contiguous
 *   dht     [N, H, Dk, Dv] f32, or NULL (zero)
 *   dq, dk  [B, T, Hg, Dk] dtype, contiguous: summed over the value heads that share them in fp32,
 *                          rounded once
 *   dv      [B, T, H, Dv]  dtype, contiguous
 *   dg      g's shape      f32, or NULL (not wanted)
 *   dh0     [N, H, Dk, Dv] f32, or NULL (not written); may be dht's buffer
 * Dk and Dv up to 128 (GDN_ERR_UNSUPPORTED beyond).  bf16 gradients are as near as fp32 sums rounded once,
 * dg and dh0 as exact as fp32 sums; dg is a difference of sums over the tokens around it, so that its error is
 * an fp32 rounding of theirs: all of it where a token's decay leaves less than 2^-24 of the state, down to
 * decays of 2^-150, from where it is 0.  Sums have a fixed order (no atomics).  Gradients
 * of tokens of a packed batch that no sequence has are not written.
 * The workspace holds a state in fp32 for every 512 tokens of a sequence (256 in f32; half of that with
 * head_decay; fewer where it is split into shorter segments): 4 Dk Dv bytes a value head, sizes rounded
 * up to 64 or 128, which is 128 bytes a token and head of 128 x 128; 8 bytes for each token and head;
 * where sequences are split, two more states a segment; and, where q/k heads are shared, every value
 * head's dq and dk in fp32, 8 Dk bytes a token and head. */
gdn_status gdn_linear_attn_bwd(const gdn_linear_desc* d, const void* q, const void* k,
                               const void* v, const float* g, const float* h0,
                               const int32_t* cu_seqlens, const void* dout, const float* dht,
                               void* dq, void* dk, void* dv, float* dg, float* dh0,
                               hipStream_t stream);

/* The same recurrence for one token of each of d->B sequences (T is 1, N is 0 or B; g [H] or [B, H]),
 * the states in a pool: sequence b reads line cache_indices[b] (b when NULL) of state [state_lines, H,
 * Dk, Dv] and writes line out_indices[b] (the line it read when NULL).  A line read from outside the
 * pool is a zero start, one written outside it is dropped.  A line that one sequence writes and
 * another reads or writes in the same call has unspecified contents.  No workspace. */
gdn_status gdn_linear_state_update(const gdn_linear_desc* d, float* state, const void* q,
                                   const void* k, const void* v, const float* g,
                                   const int32_t* cache_indices, const int32_t* out_indices,
                                   void* o, hipStream_t stream);

/* Group norm of channels-last data with an activation or a gate: the norm of a token's heads after
 * a mixing layer (positions = 1), or of a feature map's channel groups.  For sample n and group g
 * of channels / groups consecutive channels, over the sample's positions and the group's channels,
 *
 *   mean = E[x],  rstd = (E[(x - mean)^2] + eps)^-1/2,  u = (x - mean) rstd weight[c] + bias[c]
 *   y = act(u) without a gate, u act(gate) with one
 *
 * x, gate, y [samples, positions, channels] dtype (bf16 or f32), contiguous; weight, bias
 * [channels] f32 or NULL (ones, zeros); mean, rstd [samples, groups] f32, written unless NULL (the
 * backward needs them; NaN where there are no positions).  Statistics are fp32 sums about the mean.
 * Any channels, groups dividing it, up to 2^20 (GDN_ERR_UNSUPPORTED beyond, beyond 2^30 positions,
 * and beyond 2^21 (sample, group) pairs unless positions is 1 and a group has at most 1024
 * channels); pointers aligned to their element (vectors are used where 16 bytes fit). */
typedef struct gdn_norm_desc {
  int32_t samples, positions, channels, groups;
  int32_t dtype;       /* gdn_dtype of x, gate, y, dy, dx, dgate */
  int32_t activation;  /* gdn_activation */
  float eps;           /* >= 0 */
  void* workspace;     /* 256-byte aligned, as many bytes as the query gives (0 for many shapes) */
  size_t workspace_bytes;
} gdn_norm_desc;

/* Bytes of workspace of the forward (backward = 0) or the backward (1).  Host-only. */
size_t gdn_group_norm_workspace_size(const gdn_norm_desc* d, int32_t backward,
                                     gdn_status* status);

gdn_status gdn_group_norm_fwd(const gdn_norm_desc* d, const void* x, const float* weight,
                              const float* bias, const void* gate, void* y, float* mean,
                              float* rstd, hipStream_t stream);

/* Its gradient, from the forward's inputs, mean and rstd, and dy: dx, dgate (with a gate) in
 * dtype; dweight, dbias [channels] f32 sums over samples and positions (NULL: not written). */
gdn_status gdn_group_norm_bwd(const gdn_norm_desc* d, const void* x, const float* weight,
                              const float* bias, const void* gate, const float* mean,
                              const float* rstd, const void* dy, void* dx, float* dweight,
                              float* dbias, void* dgate, hipStream_t stream);

/* The norms before and after a block with its gate and residual scale, one pass over the rows: what
 * follows a block's output projection up to the next block's input.  For a row of the residual stream
 * x, the block's output h and its gate (RMS norms),
 *
 *   n = h (E[h^2] + eps)^-1/2 post_weight            (n = h without post_norm)
 *   z = n act(gate)                                  (z = n without a gate)
 *   x_out = x + residual_scale scale z               (scale NULL: ones)
 *   y = x_out (E[x_out^2] + eps)^-1/2 weight         (weight NULL: ones; y NULL: left out)
 *
 * x, x_out [rows, channels] residual_dtype; h, gate, y [rows, channels] dtype; h and gate rows
 * *_stride elements apart (0 = one after another), the others contiguous; post_weight, scale, weight
 * [channels] f32; post_rstd, rstd [rows] f32, the two norms' factors, written unless NULL (the
 * backward needs them).  Statistics are fp32 and y comes from x_out before it is rounded.  x_out may be
 * x's buffer.  h NULL: x_out is x and not written, y its norm; gate, post_weight, scale and post_norm
 * belong to h, post_weight to post_norm.  dtype bf16 or f32; residual_dtype the same, or f32 with
 * bf16.  Any channels up to 2^20, rows up to 2^30 (GDN_ERR_UNSUPPORTED beyond); pointers aligned to
 * their element (vectors are used where rows start on them).  An infinity or a NaN stays in its row. */
typedef struct gdn_block_norm_desc {
  int32_t rows, channels;
  int32_t dtype;           /* gdn_dtype of h, gate, y, dy, dh, dgate */
  int32_t residual_dtype;  /* gdn_dtype of x, x_out, dx_out, dx      */
  int32_t post_norm;       /* 0 or 1                                 */
  int32_t activation;      /* gdn_activation of the gate             */
  float eps;               /* >= 0                                   */
  float residual_scale;
  int64_t h_stride, gate_stride;
  void* workspace;         /* backward: 256-byte aligned, as many bytes as the query gives */
  size_t workspace_bytes;
} gdn_block_norm_desc;

gdn_status gdn_block_norm_fwd(const gdn_block_norm_desc* d, const void* x, const void* h,
                              const void* gate, const float* post_weight, const float* scale,
                              const float* weight, void* x_out, void* y, float* post_rstd,
                              float* rstd, hipStream_t stream);

/* Bytes of workspace gdn_block_norm_bwd needs.  Host-only. */
size_t gdn_block_norm_bwd_workspace_size(const gdn_block_norm_desc* d, gdn_status* status);

/* Its gradient, from the forward's inputs, its two factors and the gradients dx_out [rows, channels]
 * residual_dtype (NULL: zero) and dy [rows, channels] dtype (NULL: y was left out) of its outputs, one
 * of them at least: dx residual_dtype; dh (with h), dgate (with a gate) dtype; contiguous.
 * dpost_weight, dscale, dweight [channels] f32 sums over the rows in a fixed order (NULL: not
 * written). */
gdn_status gdn_block_norm_bwd(const gdn_block_norm_desc* d, const void* x, const void* h,
                              const void* gate, const float* post_weight, const float* scale,
                              const float* weight, const float* post_rstd, const float* rstd,
                              const void* dx_out, const void* dy, void* dx, void* dh, void* dgate,
                              float* dpost_weight, float* dscale, float* dweight,
                              hipStream_t stream);

/* Bytes of workspace the variant chosen by d->variant needs (for AUTO, what AUTO picks when
 * given that much).  The fused variant needs none on a dense batch; on a packed batch of
 * 2 .. 65536 sequences it asks for 4 bytes per sequence (256-byte aligned) to run them
 * longest first (an order kernel ranks them by length; the last workgroups to start are then
 * the shortest).  Given less, it runs them in index order: the same results, bit for bit.  The query cannot see cu_seqlens: a
 * descriptor with N other than 0 or B is a packed batch, one with B == 1 may be either and
 * gets the larger of the two needs, any other is a dense batch.  Host-only, no device work.
 * Returns 0 and sets *status on an invalid descriptor. */
size_t gdn_chunk_fwd_workspace_size(const gdn_desc* d, gdn_status* status);

/* The gdn_variant that gdn_chunk_fwd(d, ..., cu_seqlens, ...) runs with this descriptor and
 * workspace (AUTO resolved), or -1 if the call would be refused.  Only the nullness of
 * cu_seqlens is used; host-only, no device work. */
int32_t gdn_resolved_variant(const gdn_desc* d, const int32_t* cu_seqlens);

/* The chunk length gdn_chunk_fwd(d, ..., cu_seqlens, ...) runs with this descriptor: C for
 * the staged variant, the fused kernel's own chunk for the fused and segmented ones, 1 for
 * the recurrent one; -1 if the call would be refused.  Host-only, no device work. */
int32_t gdn_resolved_chunk(const gdn_desc* d, const int32_t* cu_seqlens);

/* The forward pass.  q, k, v, g, beta, o are required unless B*T = 0 (then every sequence
 * is empty: ht = h0, or zeros, and nothing else is touched, whatever the variant); h0 (zero
 * state), cu_seqlens (dense batch) and ht (final state not written) may be NULL.  scale multiplies o (Dk^-0.5 is the
 * usual choice).  Pointers must be device pointers aligned to 16 bytes (g, beta, cu_seqlens:
 * 4 / 2 / 4 bytes).  With stop_after = k > 0 (staged, or fused with k = 6) o and ht are
 * not written. */
gdn_status gdn_chunk_fwd(const gdn_desc* d, const void* q, const void* k, const void* v,
                         const float* g, const void* beta, const float* h0,
                         const int32_t* cu_seqlens, float scale, void* o, float* ht,
                         hipStream_t stream);

/* The decode operator with its gates made in the kernel (fused_sigmoid_gating_delta_rule,
 * the TileLang × xLLM page's section on the three core operators: the sigmoid activation,
 * the gate computation from A_log, the decay rate, and the delta-rule state update in one
 * kernel).  The page prints no formula; the reading is, per token t and value head h,
 *
 *     g_t    = -exp(A_log[h]) * softplus(a_t + dt_bias[h]),   softplus(x) = log(1 + e^x)
 *     beta_t = sigmoid(b_t) = 1 / (1 + e^-b_t)
 *
 * followed by exactly the recurrence of gdn_chunk_fwd with these g and beta, token by token
 * (the recurrent variant's kernel, the gates made in fp32 in the same kernel).
 *   a, b        [B, T, H]   d->beta_dtype (bf16 or f32): raw gate and beta inputs
 *   A_log       [H] f32     log of each head's decay rate (required)
 *   dt_bias     [H] f32     added to a before softplus, or NULL (zero)
 * Every other argument, layout and rule as for gdn_chunk_fwd (h0 and ht may be the same
 * buffer: the state is then updated in place, as a decode loop wants).  d->variant must be
 * GDN_VARIANT_AUTO or GDN_VARIANT_RECURRENT (else GDN_ERR_UNSUPPORTED); d->chunk is
 * ignored; no workspace. */
gdn_status gdn_fused_sigmoid_gating_delta_rule(const gdn_desc* d, const void* q, const void* k,
                                               const void* v, const void* a, const void* b,
                                               const float* A_log, const float* dt_bias,
                                               const float* h0, const int32_t* cu_seqlens,
                                               float scale, void* o, float* ht,
                                               hipStream_t stream);

/* How gdn_chunk_bwd(d, ..., cu_seqlens, ...) runs with this descriptor:
 * GDN_VARIANT_SEGMENTED (both sequential passes per segment), GDN_VARIANT_FUSED (the fused
 * kernel's recompute, one reverse pass per sequence), GDN_VARIANT_STAGED (the staged
 * recompute: f32), or -1 if the call would be refused.  Only the nullness of cu_seqlens is
 * used; host-only, no device work. */
int32_t gdn_chunk_bwd_resolved_variant(const gdn_desc* d, const int32_t* cu_seqlens);

/* Bytes of workspace gdn_chunk_bwd needs for this descriptor (N other than 0 or B reads as a
 * packed batch of N sequences, anything else as B dense sequences).  Host-only, no device
 * work.  Returns 0 and sets *status on an invalid or unsupported descriptor. */
size_t gdn_chunk_bwd_workspace_size(const gdn_desc* d, gdn_status* status);

/* The backward pass of gdn_chunk_fwd (the FlashQLA how-to reports forward and backward
 * speed-ups of the chunked operator, section 4.3; none of the pages prints the backward's
 * formulas).  Given the forward's inputs and the gradients of its outputs, it writes the
 * gradients of its inputs: the exact derivative of the recurrence, computed chunk by chunk
 * (C = 64) from the forward's chunk quantities, which it recomputes into the workspace
 * (nothing of a forward call is kept): T = (I + A)^-1 by the staged stages 0-4, then the
 * chunk-start states and v_new by the fused kernel (bf16), or stages 5-6 (f32).  The
 * gradients of the chunk-end states then run back through each sequence's chunks in order.
 * Few long sequences (AUTO: when segmenting pays, as for gdn_chunk_fwd's segmented variant;
 * GDN_VARIANT_SEGMENTED: always, bf16 only) run both sequential passes per segment: the
 * states from the segmented forward's maps, and the gradients by the adjoint map (a
 * segment's start gradient is M^T times its end gradient plus its own share), composed last
 * to first.  Any other variant keeps one pass per sequence.
 *   dout  [B, T, H, Dv]   qkv_dtype   gradient of o (required)
 *   dht   [N, H, Dk, Dv]  f32         gradient of ht, or NULL (zero)
 *   dq, dk [B, T, Hg, Dk] grad_dtype  the q/k heads' gradients (summed over the value heads
 *                                     that share them; fp32 sums, rounded once at the store)
 *   dv    [B, T, H, Dv]   grad_dtype
 *   dg, dbeta [B, T, H]   f32
 *   dh0   [N, H, Dk, Dv]  f32         gradient of h0, or NULL (not written)
 * Inputs, scale, cu_seqlens and their layouts as for gdn_chunk_fwd (h0 NULL = zero state).
 * Supported: bf16 with Dk = Dv in {64, 128}; f32 with Dk = Dv = 64; d->grad_dtype GDN_F32, or
 * GDN_BF16 with bf16 inputs (else GDN_ERR_UNSUPPORTED; another value: GDN_ERR_INVALID_ARG).  d->chunk and d->stop_after are ignored.  The workspace
 * (d->workspace, 256-byte aligned, gdn_chunk_bwd_workspace_size bytes) is required when
 * B*T > 0, else GDN_ERR_WORKSPACE.  Results do not depend on scheduling (no atomics).
 * Pointers are device pointers aligned to 16 bytes (g, beta, dg, dbeta, cu_seqlens: 4 / 2 /
 * 4 / 4 / 4).  With B*T = 0 only dh0 is written (= dht, or zeros). */
gdn_status gdn_chunk_bwd(const gdn_desc* d, const void* q, const void* k, const void* v,
                         const float* g, const void* beta, const float* h0,
                         const int32_t* cu_seqlens, float scale, const void* dout,
                         const float* dht, void* dq, void* dk, void* dv, float* dg,
                         float* dbeta, float* dh0, hipStream_t stream);

/* Bytes of device scratch the library holds on each GPU for gdn_chunk_fwd_noalloc. */
#define GDN_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* gdn_chunk_fwd for callers that cannot allocate device memory: code under HIP graph
 * capture, serving loops that must not call hipMalloc, harnesses that forbid it.  Same
 * arguments, checks and results as gdn_chunk_fwd, except that d->workspace and
 * d->workspace_bytes are ignored: the workspace is the library's own scratch, a static
 * device array of GDN_NOALLOC_SCRATCH_BYTES that each GPU the library runs on holds until
 * the process ends (its address is looked up on the first call on a device).  A variant
 * that needs more returns GDN_ERR_WORKSPACE; AUTO picks among what fits, as it does for
 * any workspace.  Nothing is allocated and nothing needs clearing between calls.  Every
 * call on one GPU shares that GPU's scratch: calls that overlap on one GPU (other streams,
 * other host threads) race and give unspecified results.  stop_after must be 0
 * (GDN_ERR_INVALID_ARG otherwise): stage buffers in the scratch are out of the caller's
 * reach. */
gdn_status gdn_chunk_fwd_noalloc(const gdn_desc* d, const void* q, const void* k,
                                 const void* v, const float* g, const void* beta,
                                 const float* h0, const int32_t* cu_seqlens, float scale,
                                 void* o, float* ht, hipStream_t stream);

/* Where intermediate `buf` lives inside the workspace of a stage-stop call (offset and size
 * in bytes), for stage-by-stage inspection (the page's section 7.4 debugging mode): the
 * staged layout at C, or, for GDN_VARIANT_FUSED with stop_after = 6, the fused stop's
 * layout at 64-token chunks, where the buffers it does not write have size 0. */
gdn_status gdn_stage_buffer(const gdn_desc* d, int32_t buf, size_t* offset, size_t* bytes);

/* Static, human-readable text for a status code. */
const char* gdn_status_string(gdn_status s);

/* Library version: major * 10000 + minor * 100 + patch. */
int32_t gdn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
