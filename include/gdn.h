/*
 * gdn.h - C interface of the GB300 (sm_103a) gated delta-rule library.
 *
 * The method: a linear-attention state S (V x K per value head) evolves per
 * token t as
 *     S_t = S_{t-1} * D_t * (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,
 *     o_t = scale * S_t q_t,
 * with D_t = exp(g_t) * I (GDN, one log-gate per token and head) or
 * D_t = diag(exp(g_t[0..K))) (KDA, one log-gate per token, head and key
 * channel).  The token form (decay, pred = S k, delta = beta (v - pred),
 * S += delta k^T, o = S q) is the one of the FlashInfer page
 * gdn_decode_bf16_state.py (per-token helpers); the chunked form with BT = 64
 * token chunks follows the sglang page fla/chunk_fwd.py (fused KK^T + solve
 * kernel, Steps 1-5, and chunk_gated_delta_rule_fwd_intra), the KDA page
 * _fla/ops/common/chunk_h.py (chunk_fwd_kernel_h, chunk_fwd_h) and the vLLM
 * kimi_k3 kda/chunk_intra page (chunk_kda_fwd_kernel_inter_solve_fused).
 *
 * Conventions shared by every entry point
 *  - Memory: every tensor pointer is a DEVICE pointer owned by the caller.
 *    The library never allocates, frees or retains device memory; outputs are
 *    written in place.  Tensors are dense, row-major, last index fastest, in
 *    the layouts given per argument.  Every tensor pointer must be 16-byte
 *    aligned (GDN_ERR_MISALIGNED otherwise).
 *  - Streams: work is enqueued on the caller's stream (NULL = the legacy
 *    default stream) and the call returns without waiting for it.
 *  - Errors: every call returns a gdn_status_t and never throws, exits or
 *    prints.  Argument errors are found on the host before anything is
 *    enqueued (nothing is written then).  Errors that only the device can see
 *    (bad cu_seqlens, bad slot index, a bounded wait that ran out) are
 *    recorded in a device-side error word, which gdn_check_device_error()
 *    reads and clears.  gdn_last_error_message() describes the last host-side
 *    failure of the calling thread.
 *  - Log-gates are natural logarithms (exp, not exp2).
 */
#ifndef GDN_GB300_H
#define GDN_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t / CUstream. */
typedef struct CUstream_st *gdn_stream_t;

typedef enum gdn_status {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARG = 1,  /* NULL required pointer, bad size or flag    */
  GDN_ERR_UNSUPPORTED = 2,  /* valid request this library does not serve */
  GDN_ERR_MISALIGNED = 3,   /* a tensor pointer is not 16-byte aligned    */
  GDN_ERR_WORKSPACE = 4,    /* workspace smaller than *_workspace_size     */
  GDN_ERR_CUDA = 5,         /* a CUDA runtime call failed                  */
  GDN_ERR_TIMEOUT = 6,      /* device: a bounded wait gave up              */
  GDN_ERR_BAD_SEQLENS = 7,  /* device: cu_seqlens not rising from 0 to T   */
  GDN_ERR_BAD_SLOT = 8,     /* device: a slot index outside [0, pool)      */
  GDN_ERR_BOUNDS = 9        /* device, checked builds only: an index range a
                               kernel derived falls outside its tensor; the
                               CTA skips its work                          */
} gdn_status_t;

typedef enum gdn_dtype {
  GDN_F32 = 0,   /* float32 q, k, v, o  */
  GDN_BF16 = 1   /* bfloat16 q, k, v, o */
} gdn_dtype_t;

/*
 * Chunked forward with one scalar log-gate per token and value head (GDN).
 * Shapes follow chunk_gated_delta_rule_fwd_intra (sglang fla/chunk_fwd.py)
 * and chunk_fwd_h (KDA _fla/ops/common/chunk_h.py):
 *   q, k   [B, T, Hg, K]  dtype       key/query heads; value head h reads
 *                                     key head h / (H / Hg)
 *   v, o   [B, T, H, V]   dtype       o is written, in float32 instead
 *                                     when o_fp32 = 1 (the same result
 *                                     before its rounding to dtype: with
 *                                     o_fp32 = 0 and bf16, o is exactly the
 *                                     round-to-nearest-even of that value)
 *   g      [B, T, H]      float32     natural-log gate per token; with
 *                                     g_is_cumsum = 1 it is instead the
 *                                     inclusive cumulative sum inside each
 *                                     64-token chunk (chunks counted from
 *                                     each sequence's first token).  The
 *                                     sums are held in float32: a gate of
 *                                     -1e4 costs the tokens behind it in
 *                                     its chunk 5e-3 of o, -80 3e-5, and
 *                                     -infinity or the lowest float leaves
 *                                     NaN; -104 forgets as much as those
 *                                     (e^-104 is zero in float32)
 *   beta   [B, T, H]      float32
 *   h0     [N, H, K, V]   float32     initial state h = S^T, NULL = zeros
 *   ht     [N, H, K, V]   float32     final state, NULL = not returned
 *   state_v_first = 1     h0 and ht hold every state transposed,
 *                                     [N, H, V, K] (S itself; the chunk_h
 *                                     page's state_v_first); 0 = [K, V]
 *   cu_seqlens [N + 1]    int32       NULL: N = B sequences of T tokens.
 *                                     Else B must be 1 and sequence n is
 *                                     tokens cu_seqlens[n] .. cu_seqlens[n+1]
 *                                     (0 = cu_seqlens[0] <= ... <= cu_seqlens[N]
 *                                     = T, checked on the device)
 * Limits: 1 <= K <= 128, V >= 1, chunk_size == 64, H % Hg == 0, N and H at
 * most 65535 (GDN_ERR_UNSUPPORTED otherwise).  With T == 0
 * nothing per token is read or written, so q, k, v, g, beta and o may be NULL
 * (ht = h0, or zeros).
 * scale <= 0 selects 1/sqrt(K).
 * Workspace: bf16 inputs with K == 128 and V a multiple of 32 up to 128 run on
 * the tensor cores and need `workspace` (device, 256-byte aligned,
 * caller-owned, contents irrelevant before and after the call) of at least
 * gdn_chunk_workspace_size() bytes, else GDN_ERR_WORKSPACE.  Every other
 * shape runs the exact fp32 CUDA-core kernel and needs none.
 * Segment-parallel state pass (tensor-core path; `segments`): the chunk
 * recurrence h <- M_c h + B_c is affine in h, so with S >= 2 every sequence
 * is cut into S runs of ceil(chunks / S) chunks that are all processed at
 * once -- each from a zero state and on the identity, which gives the run's
 * map (M, B) -- then combined in order (start of run s + 1 = M start_s + B)
 * and run again from their true starts, writing o.  The sequential part
 * shrinks from `chunks` to about 2 chunks / S steps, at about three times
 * the work; it pays when the sequences' own chains (V / 32 per head and
 * sequence) leave most SMs idle.  0 lets the library choose (1 unless that
 * holds); the fp32 CUDA-core kernel ignores it.  1 <= segments <= 64 and
 * N * segments <= 65535, else GDN_ERR_UNSUPPORTED.
 */
typedef struct gdn_chunk_args {
  int32_t dtype;               /* gdn_dtype_t of q, k, v, o */
  const void *q, *k, *v;
  const float *g, *beta;
  const float *h0;
  float *ht;
  void *o;
  const int32_t *cu_seqlens;
  int32_t B, T, H, Hg, K, V, N;
  int32_t chunk_size;
  int32_t g_is_cumsum;
  int32_t state_v_first;       /* 1: h0, ht are [N, H, V, K] instead of [N, H, K, V] */
  int32_t o_fp32;              /* 1: o is float32 whatever dtype is; 0: o has dtype */
  int32_t segments;            /* state pass: 0 = library's choice, 1 = one chain per
                                  sequence, 2..64 = segment-parallel (see above) */
  float scale;
  void *workspace;
  size_t workspace_bytes;
} gdn_chunk_args;

/* Bytes of workspace gdn_chunk_fwd needs for these arguments (0 when the
 * CUDA-core kernel serves them).  Reads only sizes, dtype and whether
 * cu_seqlens is NULL. */
gdn_status_t gdn_chunk_workspace_size(const gdn_chunk_args *args, size_t *bytes);

/* The segment count gdn_chunk_fwd would use for the state pass with these
 * arguments (args->segments, or the library's choice when it is 0; 1 when
 * the exact fp32 CUDA-core kernel serves them).  Reads only sizes, dtype,
 * segments and whether cu_seqlens is NULL. */
gdn_status_t gdn_chunk_segment_count(const gdn_chunk_args *args, int32_t *segments);

/* Enqueue the GDN chunked forward (gate cumsum, intra-chunk (I+A)^-1 with the
 * WY vectors w, u, the sequential inter-chunk state pass and the output) on
 * `stream`.  Writes o and, if given, ht. */
gdn_status_t gdn_chunk_fwd(const gdn_chunk_args *args, gdn_stream_t stream);

/*
 * The same forward end to end from HOST memory: q, k, v, g, beta, h0,
 * cu_seqlens are read from and o, ht written to host buffers (pinned memory
 * lets the copies run asynchronously and at full speed; pageable memory is
 * accepted).  Shapes, limits and NULL rules are those of gdn_chunk_fwd.
 * `workspace` is a DEVICE buffer on the current device, 256-byte aligned,
 * caller-owned, of at least gdn_chunk_host_workspace_size() bytes: it takes
 * device copies of the inputs and outputs and the kernels' scratch.
 * The call enqueues everything behind the work already on `stream` and
 * returns; o and ht are complete in host memory when `stream` has completed
 * (e.g. cudaStreamSynchronize).  Host buffers must stay valid and unchanged
 * until then.  Inside, the problem is cut into pieces of whole 64-token
 * chunks along time (sequences of more than 704 tokens; the pieces shrink
 * towards the end) or into ranges of whole sequences, and each piece's host->device copies, kernels
 * and device->host copies run on an internal copy-in stream, `stream` and an
 * internal copy-out stream, so the copies of one piece overlap the kernels of
 * its neighbours.  The state pass runs one chain per sequence (`segments`
 * is ignored), and the results equal gdn_chunk_fwd's with segments = 1 bit
 * for bit: a time cut hands the fp32 state of the chunkwise recurrence (Gated
 * Delta Networks, section 3) from one piece to the next exactly as the
 * kernels carry it between chunks.
 * Errors: argument errors as gdn_chunk_fwd, plus GDN_ERR_INVALID_ARG when an
 * input or output pointer is device memory, GDN_ERR_WORKSPACE when the
 * workspace is missing, too small or not device memory, GDN_ERR_BAD_SEQLENS
 * (returned by the call itself) when cu_seqlens does not rise from 0 to T.
 * With cu_seqlens the call copies offsets rebased per piece from pageable
 * memory, so it cannot be captured into a CUDA graph; without, it can.
 * Calls from several host threads are serialised inside the library.
 */
gdn_status_t gdn_chunk_fwd_host(const gdn_chunk_args *args, gdn_stream_t stream);

/*
 * Chunk state pass of gated linear attention (KDA _fla/ops/common/chunk_h.py:
 * chunk_fwd_kernel_h / chunk_fwd_h, "h += k^T v" with an optional decay).
 * For every sequence n and head h the state h [K, V] starts at h0 (or zeros)
 * and takes, token by token,
 *     h <- Dk_t h Dv_t + k_t v_t^T
 * where the decay depends on `gate` (natural-log gates):
 *   GDN_GATE_NONE      Dk = Dv = I                       gate_values NULL
 *   GDN_GATE_G         Dk = e^{r_t} I                    gate_values [B,T,H]
 *   GDN_GATE_G_GAMMA   Dk = e^{gamma_h} I, every token   gate_values [H]
 *   GDN_GATE_GK        Dk = diag(e^{r_t[:]}) (keys)      gate_values [B,T,H,K]
 *   GDN_GATE_GV        Dv = diag(e^{r_t[:]}) (values)    gate_values [B,T,H,V]
 * The per-token gates are given as the page's kernel takes them: inclusive
 * cumulative sums of r_t inside each 64-token chunk (chunks counted from each
 * sequence's first token); g_gamma is the per-token rate itself.
 *   k [B,T,H,K], v [B,T,H,V]   dtype (GDN_F32 or GDN_BF16)
 *   h0, ht [N,H,K,V]           float32, NULL = zeros / not returned
 *   hs [C,H,K,V]               hs_dtype (GDN_F32 or GDN_BF16): the state at the
 *                              start of every split (split_size tokens, a
 *                              multiple of 64; 0 = 64: every chunk), sequence
 *                              after sequence (sequence n contributes
 *                              ceil(len_n / split_size) entries; B equal
 *                              sequences: [B, ceil(T/split_size), ...]);
 *                              NULL = not returned; num_chunks = C, its capacity
 *   cu_seqlens [N + 1] int32   as gdn_chunk_fwd (device memory; checked on the
 *                              device, GDN_ERR_BAD_SEQLENS also when the chunks
 *                              do not fit num_chunks)
 *   state_v_first = 1          every state tensor (h0, ht, hs) holds each
 *                              state transposed, [V, K] (the page's
 *                              state_v_first); the arithmetic is unchanged
 * Limits: 1 <= K <= 128, K and V multiples of 8, chunk_size == 64, N and H at
 * most 65535.
 * Arithmetic in fp32 (bf16 inputs are widened).  Nothing is allocated; no
 * workspace.
 */
typedef enum gdn_gate_kind {
  GDN_GATE_NONE = 0,
  GDN_GATE_G = 1,
  GDN_GATE_G_GAMMA = 2,
  GDN_GATE_GK = 3,
  GDN_GATE_GV = 4
} gdn_gate_kind_t;

typedef struct gdn_state_args {
  int32_t dtype;               /* gdn_dtype_t of k, v */
  const void *k, *v;
  int32_t gate;                /* gdn_gate_kind_t */
  const float *gate_values;
  const float *h0;
  float *ht;
  void *hs;
  int32_t hs_dtype;            /* gdn_dtype_t of hs */
  const int32_t *cu_seqlens;
  int32_t B, T, H, K, V, N;
  int32_t chunk_size;
  int64_t num_chunks;
  int32_t split_size;          /* tokens between stored states; 0 = chunk_size */
  int32_t state_v_first;       /* 1: h0, ht, hs are [.., V, K] instead of [.., K, V] */
} gdn_state_args;

/* Enqueue the chunk state pass on `stream`. */
gdn_status_t gdn_chunk_state_fwd(const gdn_state_args *args, gdn_stream_t stream);

/*
 * Backward state pass (KDA _fla/ops/common/chunk_h.py: chunk_bwd_kernel_dh /
 * chunk_bwd_dh): for the recurrence of gdn_chunk_state_fwd with outputs
 * o_t = scale S_t^T q_t (S_t the state after token t), the gradient
 * G = dL/dS of a loss with dL/do_t = do_t, going from the last token back:
 *     G <- G + scale q_t do_t^T,   then   G <- decay_t^T(G)
 * starting from dht (or zeros).  Per query head hq (gate head hq / (HQ / H)):
 *   q [B,T,HQ,K], do [B,T,HQ,V]  dtype (GDN_F32 or GDN_BF16)
 *   gate, gate_values            as gdn_chunk_state_fwd, with H heads
 *   dht, dh0 [N,HQ,K,V]          float32, NULL = zeros / not returned
 *   dh [C,HQ,K,V]                dh_dtype: the gradient with respect to the
 *                                state at the end of the first chunk of every
 *                                split (before that chunk's tokens are folded
 *                                in; split_size as gdn_chunk_state_fwd, 0 = every
 *                                chunk), sequence after sequence; NULL = not
 *                                returned; num_chunks = C
 *   scale                        <= 0 selects 1/sqrt(K)
 * Limits, errors and the rest as gdn_chunk_state_fwd; HQ % H == 0.
 */
typedef struct gdn_state_bwd_args {
  int32_t dtype;               /* gdn_dtype_t of q, do */
  const void *q, *do_;
  int32_t gate;                /* gdn_gate_kind_t */
  const float *gate_values;
  const float *dht;
  float *dh0;
  void *dh;
  int32_t dh_dtype;            /* gdn_dtype_t of dh */
  const int32_t *cu_seqlens;
  int32_t B, T, HQ, H, K, V, N;
  int32_t chunk_size;
  int64_t num_chunks;
  float scale;
  int32_t split_size;          /* tokens between stored gradients; 0 = chunk_size */
  int32_t state_v_first;       /* 1: dht, dh0, dh are [.., V, K] instead of [.., K, V] */
} gdn_state_bwd_args;

/* Enqueue the backward state pass on `stream`. */
gdn_status_t gdn_chunk_state_bwd(const gdn_state_bwd_args *args, gdn_stream_t stream);

/* Bytes of device workspace gdn_chunk_fwd_host needs for these arguments.
 * Reads sizes, dtype and, when given, the host array cu_seqlens. */
gdn_status_t gdn_chunk_host_workspace_size(const gdn_chunk_args *args, size_t *bytes);

/*
 * Gradient of gdn_chunk_fwd: of a loss with dL/do and dL/dht given, with respect to q, k, v,
 * g, beta and h0.  Everything the forward computed is formed again from its inputs; nothing
 * of that call is kept.
 *   q, k, dq, dk  [B, T, Hg, K]   dtype    dq and dk summed over the value heads that share
 *                                          the key head
 *   v, do, dv     [B, T, H, V]    dtype
 *   g, beta, dg, dbeta [B, T, H]  float32  dg is the gradient of g as given: of the per-token
 *                                          gate, or of the chunk-local sum (g_is_cumsum = 1)
 *   h0, dht, dh0  [N, H, K, V]    float32  ([N, H, V, K] with state_v_first = 1); NULL =
 *                                          zeros / zeros / not returned
 *   cu_seqlens    [N + 1]         int32    as gdn_chunk_fwd; with bad offsets nothing is
 *                                          written
 * A per-token gate may be anything down to -infinity (the state is forgotten: e^g is zero below
 * -104), although gdn_chunk_fwd wants it above some -1e2; a chunk-local sum has to be finite.
 * A NaN or an infinity in v or do may reach every token of its chunk and, of its sequence,
 * those that its state or the state's gradient reaches; other sequences and heads (but for dq
 * and dk of its key head) are as without it.
 * With T == 0 the per-token arrays may be NULL (dh0 = dht, or zeros).  Outputs must not
 * overlap inputs.  A sum over heads, tokens or channels always runs in the same order, so
 * results do not change from run to run.
 * Accuracy: float32 inputs are taken in float32 throughout.  With bfloat16 inputs, K and V
 * multiples of 8 and V <= 128 the products run on the tensor cores, whose operands carry
 * float32 values (states, their gradients, corrected values, T and P) as two bfloat16 pieces:
 * each is off by up to 2^-17 of itself (below 6e-36 by 2^-134), sums are float32, and dq, dk
 * and dv are rounded once (float32 results are within 1e-5 of their norm, those of a few tokens,
 * whose errors do not average out, within 3e-5; gates that forget, as many as there are,
 * included).
 * Limits: as gdn_chunk_fwd, and V <= 2^20.  scale <= 0 selects 1/sqrt(K).
 * Workspace: gdn_chunk_bwd_workspace_size() bytes, device memory, 256-byte aligned: for every
 * chunk of 64 tokens and value head A, T, P, the corrected values and their gradients, the
 * state and its gradient (241 KB with K = V = 128).
 */
typedef struct gdn_chunk_bwd_args {
  int32_t dtype;               /* gdn_dtype_t of q, k, v, do, dq, dk, dv */
  const void *q, *k, *v;
  const float *g, *beta;
  const float *h0;
  const void *do_;
  const float *dht;
  void *dq, *dk, *dv;
  float *dg, *dbeta;
  float *dh0;
  const int32_t *cu_seqlens;
  int32_t B, T, H, Hg, K, V, N;
  int32_t chunk_size;
  int32_t g_is_cumsum;
  int32_t state_v_first;
  float scale;
  void *workspace;
  size_t workspace_bytes;
} gdn_chunk_bwd_args;

/* Bytes of workspace gdn_chunk_bwd needs; reads only sizes, dtype and whether cu_seqlens is
 * NULL. */
gdn_status_t gdn_chunk_bwd_workspace_size(const gdn_chunk_bwd_args *args, size_t *bytes);
gdn_status_t gdn_chunk_bwd(const gdn_chunk_bwd_args *args, gdn_stream_t stream);

/*
 * Chunked forward with one log-gate per token, value head and key channel
 * (KDA).  Shapes follow chunk_kda_fwd_kernel_inter_solve_fused (vLLM kimi_k3
 * kda/chunk_intra page):
 *   q, k   [B, T, H, K]   dtype       value head hv reads key head hv / (HV / H)
 *   v, o   [B, T, HV, V]  dtype       (o float32 with o_fp32 = 1, as for GDN)
 *   g      [B, T, HV, K]  float32     chunk-local inclusive cumulative sum of
 *                                     the per-channel log-gates when
 *                                     g_is_cumsum = 1 (as that kernel takes
 *                                     it), raw per-token log-gates when 0
 *   beta   [B, T, HV]     float32
 *   h0, ht [N, HV, K, V]  float32     as for GDN ([N, HV, V, K] with
 *                                     state_v_first = 1)
 *   cu_seqlens            as for GDN
 * Limits: 1 <= K <= 128, V >= 1, chunk_size == 64, HV % H == 0, N and HV at
 * most 65535.  With T == 0
 * q, k, v, g, beta and o may be NULL (ht = h0, or zeros).
 * Workspace: as for GDN (tensor cores for bf16, K == 128, V % 32 == 0,
 * V <= 128; kda_chunk_workspace_size() bytes).
 */
typedef struct kda_chunk_args {
  int32_t dtype;
  const void *q, *k, *v;
  const float *g, *beta;
  const float *h0;
  float *ht;
  void *o;
  const int32_t *cu_seqlens;
  int32_t B, T, H, HV, K, V, N;
  int32_t chunk_size;
  int32_t g_is_cumsum;
  int32_t state_v_first;       /* 1: h0, ht are [N, HV, V, K] instead of [N, HV, K, V] */
  int32_t o_fp32;              /* 1: o is float32 whatever dtype is; 0: o has dtype */
  int32_t segments;            /* as gdn_chunk_args.segments */
  float scale;
  void *workspace;
  size_t workspace_bytes;
} kda_chunk_args;

gdn_status_t kda_chunk_workspace_size(const kda_chunk_args *args, size_t *bytes);
gdn_status_t kda_chunk_fwd(const kda_chunk_args *args, gdn_stream_t stream);

/*
 * Decode step for T = 1..4 new tokens per batch entry against a pooled
 * bfloat16 state, updated in place (FlashInfer gdn_decode_bf16_state.py,
 * public gated_delta_rule and compute_single_gate):
 *   q, k     [B, T, H, K]     bf16
 *   v        [B, T, HV, V]    bf16      value head hv reads key head hv/(HV/H)
 *   a, b     [B, T, HV]       bf16      gate inputs
 *   A_log    [HV]             float32
 *   dt_bias  [HV]             float32
 *   state    [pool, HV, V, K] bf16      K fastest; slot slot_indices[b] is
 *                                       read, advanced by the T tokens in
 *                                       float32 and written back once
 *                                       (round to nearest even)
 *   slot_indices [B]          int32     NULL = identity (needs pool >= B).
 *                                       Slots must be distinct; a slot
 *                                       outside [0, pool) records
 *                                       GDN_ERR_BAD_SLOT and that entry's o
 *                                       is written as zeros.
 *   o        [B, T, HV, V]    bf16      (float32 when o_fp32 = 1: the same
 *                                       value before its rounding to bf16)
 *   new_state_f32 [B, HV, V, K] float32 or NULL: when given, entry b's
 *                                       updated state in float32, the value
 *                                       whose round-to-nearest-even the pool
 *                                       receives (NULL = not written)
 * Per token: g = -exp(A_log) * softplus(a + dt_bias) with
 *   softplus(x) = log(1 + exp(beta_sp x)) / beta_sp if beta_sp x <= threshold
 *   else x; beta = sigmoid(b); if use_qk_l2norm, q and k are divided by
 *   sqrt(sum(x^2) + eps); q is multiplied by scale.
 * Limits: K == V == 128, 1 <= T <= 4, HV % H == 0.  scale <= 0 selects
 * 1/sqrt(K); softplus_beta <= 0 selects 1; eps < 0 selects 1e-6.
 */
typedef struct gdn_decode_args {
  const void *q, *k, *v;
  const void *a, *b;
  const float *A_log, *dt_bias;
  void *state;
  const int32_t *slot_indices;
  void *o;
  float *new_state_f32;
  int32_t B, T, H, HV, K, V, pool;
  int32_t use_qk_l2norm;
  int32_t o_fp32;
  float scale, softplus_beta, softplus_threshold, eps;
} gdn_decode_args;

gdn_status_t gdn_decode(const gdn_decode_args *args, gdn_stream_t stream);

/*
 * Short causal depthwise convolution, the operator in front of the recurrences:
 * every channel d of a sequence is filtered along time with W taps,
 *     p_t[d] = bias[d] + sum_{i<W} weight[d][i] x_{t-W+1+i}[d],   y = act(p),
 * where the W - 1 rows before the sequence's first token come from h0 (oldest
 * first; zeros if NULL) and act is the identity or SiLU, p / (1 + e^-p).
 *   x, y     [B, T, D]       dtype    token rows x_stride / y_stride elements
 *                                     apart and batch rows x_batch_stride /
 *                                     y_batch_stride apart (the channels are
 *                                     dense), so that x may be a column range
 *                                     of a wider projection (any element may
 *                                     be its first); y must not overlap x
 *   weight   [D, W]          weight_dtype (GDN_F32, or dtype)
 *   bias     [D]             weight_dtype, NULL = none
 *   h0, ht   [N, W - 1, D]   dtype    rows before the first token / the last
 *                                     W - 1 rows (of h0 and x together), NULL =
 *                                     zeros / not returned; ht must not overlap
 *                                     h0
 *   cu_seqlens [N + 1]       int32    as gdn_chunk_fwd; with bad offsets
 *                                     (GDN_ERR_BAD_SEQLENS) nothing is written
 * Limits: 2 <= W <= 4, T <= 2^31 - 256.  Sums in float32, one rounding at the
 * end.  SiLU and its derivative come from the hardware's fast exponential and
 * reciprocal, for float32 too: off by a few 2^-23, and for negative p by another
 * |p| 2^-23 of values that are themselves near |p| e^p.  A stride must be at
 * least D.
 */
typedef struct short_conv_args {
  int32_t dtype;               /* gdn_dtype_t of x, y, h0, ht */
  int32_t weight_dtype;        /* gdn_dtype_t of weight, bias */
  const void *x;
  const void *weight, *bias;
  const void *h0;
  void *ht;
  void *y;
  const int32_t *cu_seqlens;
  int64_t x_stride, x_batch_stride, y_stride, y_batch_stride;
  int32_t B, T, D, W, N;
  int32_t silu;                /* 1: SiLU, 0: identity */
} short_conv_args;

gdn_status_t short_conv_fwd(const short_conv_args *args, gdn_stream_t stream);

/*
 * Gradient of short_conv_fwd: with dp_t = dy_t act'(p_t),
 *     dx_t = sum_i weight[i] dp_{t+W-1-i}   (tokens of the same sequence), plus
 *            the row of dht that x_t became, if it did,
 *     dh0  = the same sums at the W - 1 rows before the sequence,
 *     dweight[i] = sum_t dp_t x_{t-W+1+i},   dbias = sum_t dp_t.
 *   dy, x    [B, T, D]       dtype    strided as x above
 *   dx       [B, T, D]       dtype    strided; must not overlap x or dy
 *   h0, dht, dh0 [N, W-1, D] dtype    NULL = zeros / zeros / not returned
 *   dweight  [D, W], dbias [D] float32, NULL = not returned
 * The sums over tokens run in a fixed order (float32 partial sums in
 * `workspace`, 16-byte aligned, short_conv_bwd_workspace_size() bytes), so
 * results do not change from run to run.  The rest as short_conv_fwd.
 */
typedef struct short_conv_bwd_args {
  int32_t dtype;               /* gdn_dtype_t of dy, x, dx, h0, dht, dh0 */
  int32_t weight_dtype;        /* gdn_dtype_t of weight, bias */
  const void *dy, *x;
  const void *weight, *bias;
  const void *h0, *dht;
  void *dx;
  float *dweight, *dbias;
  void *dh0;
  const int32_t *cu_seqlens;
  int64_t dy_stride, dy_batch_stride, x_stride, x_batch_stride, dx_stride, dx_batch_stride;
  int32_t B, T, D, W, N;
  int32_t silu;
  void *workspace;
  size_t workspace_bytes;
} short_conv_bwd_args;

/* Bytes of workspace short_conv_bwd needs; reads sizes, strides, dtype, the
 * alignment of dy, x and dx, and whether cu_seqlens, dweight and dbias are NULL. */
gdn_status_t short_conv_bwd_workspace_size(const short_conv_bwd_args *args, size_t *bytes);
gdn_status_t short_conv_bwd(const short_conv_bwd_args *args, gdn_stream_t stream);

/*
 * short_conv_fwd for T = 1..4 new tokens per batch entry against pooled
 * states, updated in place:
 *   x, y     [B, T, D]          dtype  strided as above
 *   state    [pool, W - 1, D]   dtype  the last W - 1 rows of each request,
 *                                      oldest first
 *   slot_indices [B]            int32  as gdn_decode (NULL = identity; distinct;
 *                                      a slot outside [0, pool) records
 *                                      GDN_ERR_BAD_SLOT and that entry's y is
 *                                      written as zeros)
 */
typedef struct short_conv_decode_args {
  int32_t dtype;               /* gdn_dtype_t of x, y, state */
  int32_t weight_dtype;        /* gdn_dtype_t of weight, bias */
  const void *x;
  const void *weight, *bias;
  void *state;
  const int32_t *slot_indices;
  void *y;
  int64_t x_stride, x_batch_stride, y_stride, y_batch_stride;
  int32_t B, T, D, W, pool;
  int32_t silu;
} short_conv_decode_args;

gdn_status_t short_conv_decode(const short_conv_decode_args *args, gdn_stream_t stream);

/*
 * Selective state space scan over prompts, one scalar decay per token and head
 * (the recurrence of gdn_chunk_fwd without its delta term, with step sizes, a
 * skip term and a gate).  Per sequence and head, with the state h [V, K]
 * starting at h0 (or zeros):
 *     s_t = softplus(dt_t + dt_bias)   (dt_softplus = 1; else dt_t + dt_bias)
 *     h_t = e^(-e^A_log s_t) h_{t-1} + s_t x_t Bm_t^T
 *     y_t = h_t Cm_t + D x_t,   then y_t *= silu(z_t) if z is given
 * with softplus(v) = log(1 + e^v), v itself above 20.
 *   x, z, y  [B, T, H, V]   dtype    z NULL = no gate; y float32 when
 *                                    y_fp32 = 1
 *   Bm, Cm   [B, T, Hg, K]  dtype    head h reads group h / (H / Hg)
 *   dt       [B, T, H]      dt_dtype (GDN_F32, or dtype)
 *   A_log, D, dt_bias [H]   float32  D and dt_bias NULL = zeros
 *   h0, ht   [N, H, V, K]   float32  NULL = zeros / not returned
 *   cu_seqlens [N + 1]      int32    as gdn_chunk_fwd; with bad offsets nothing
 *                                    is written
 * x, z, Bm, Cm, dt and y have token rows *_stride elements apart and batch rows
 * *_batch_stride apart; within a row the last two dimensions are dense, so all
 * of them may be column ranges of wider buffers, starting at any element.
 * Outputs must not overlap inputs.
 * Accuracy: states are float32 throughout.  y is float32 arithmetic, rounded once,
 * but where the tensor cores take the call (dtype GDN_BF16, K <= 128, K and V
 * multiples of 8, 16-byte aligned rows): there what h_t and the weights of the
 * tokens x_j, j <= t, are multiplied with enters to 16 bits, so that y is off by at
 * most 2^-16 of the sum of its terms' magnitudes (2e-6 in norm), also with y_fp32.
 * An Inf or NaN in x reaches its row of h and of y from its token on, and nothing
 * else; that y may be NaN where the recurrence has an infinity.  Step sizes below
 * zero let h grow: the sums of -e^A_log s over 128 tokens should then stay within
 * +-80.
 * Limits: 1 <= K <= 256, H % Hg == 0, N and H at most 65535, T <= 2^31 - 256.
 * Segments: a sequence longer than `segment_tokens` (a multiple of 128; 0 = the
 * library's choice, whole sequences when their number fills the GPU) is cut
 * into segments of that many tokens that are processed at once: first each
 * one's last state from zero, then each from its start state.
 * Workspace: ssm_chunk_workspace_size() bytes (0 when no sequence is cut),
 * device memory, 256-byte aligned.
 */
typedef struct ssm_chunk_args {
  int32_t dtype;               /* gdn_dtype_t of x, z, Bm, Cm, y */
  int32_t dt_dtype;            /* gdn_dtype_t of dt */
  const void *x, *z, *Bm, *Cm, *dt;
  const float *A_log, *D, *dt_bias;
  const float *h0;
  float *ht;
  void *y;
  const int32_t *cu_seqlens;
  int64_t x_stride, x_batch_stride, z_stride, z_batch_stride;
  int64_t Bm_stride, Bm_batch_stride, Cm_stride, Cm_batch_stride;
  int64_t dt_stride, dt_batch_stride, y_stride, y_batch_stride;
  int32_t B, T, H, Hg, K, V, N;
  int32_t dt_softplus;
  int32_t y_fp32;              /* 1: y is float32 whatever dtype is; 0: y has dtype */
  int32_t segment_tokens;      /* longest run of tokens taken in sequence; 0 = choose */
  void *workspace;
  size_t workspace_bytes;
} ssm_chunk_args;

/* Bytes of workspace ssm_chunk_fwd needs; reads sizes, strides, dtype,
 * segment_tokens, pointers' alignment and whether cu_seqlens is NULL. */
gdn_status_t ssm_chunk_workspace_size(const ssm_chunk_args *args, size_t *bytes);
gdn_status_t ssm_chunk_fwd(const ssm_chunk_args *args, gdn_stream_t stream);

/*
 * The scan for T = 1..4 new tokens per batch entry against pooled states,
 * updated in place (float32 arithmetic, one rounding when state_dtype is
 * GDN_BF16):
 *   x, z, y  [B, T, H, V], Bm, Cm [B, T, Hg, K], dt [B, T, H]  as above
 *   state    [pool, H, V, K]   state_dtype   K fastest
 *   slot_indices [B]           int32         as gdn_decode
 * Limits: 8 <= K <= 256, K % 8 == 0, H % Hg == 0.
 */
typedef struct ssm_decode_args {
  int32_t dtype;               /* gdn_dtype_t of x, z, Bm, Cm, y */
  int32_t dt_dtype;            /* gdn_dtype_t of dt */
  int32_t state_dtype;         /* gdn_dtype_t of state */
  const void *x, *z, *Bm, *Cm, *dt;
  const float *A_log, *D, *dt_bias;
  void *state;
  const int32_t *slot_indices;
  void *y;
  int64_t x_stride, x_batch_stride, z_stride, z_batch_stride;
  int64_t Bm_stride, Bm_batch_stride, Cm_stride, Cm_batch_stride;
  int64_t dt_stride, dt_batch_stride, y_stride, y_batch_stride;
  int32_t B, T, H, Hg, K, V, pool;
  int32_t dt_softplus;
  int32_t y_fp32;
} ssm_decode_args;

gdn_status_t ssm_decode(const ssm_decode_args *args, gdn_stream_t stream);

/*
 * Norm over groups of channels of every token, with an activation or a gate: what
 * stands between a recurrence and its output projection (a group is a head there),
 * and group norm, channels last, where every token is a sample of its own (its
 * statistics reach no other token, so that the layer stays causal).  Per token and
 * group of W = D / groups channels:
 *     u = x, or x act(z) with gate_first = 1
 *     n = (u - mean(u)) / sqrt(mean((u - mean(u))^2) + eps)     center = 1
 *     n = u / sqrt(mean(u^2) + eps)                             center = 0
 *     m = n weight + bias
 *     y = m act(z) with z, act(m) without z, m with gate_first
 *   x, z, y  [B, T, D]      dtype    strided as in short_conv_fwd (z NULL = none);
 *                                    y must not overlap x or z
 *   weight, bias            weight_dtype (GDN_F32, or dtype): [D], or [D / groups] for
 *                                    all groups with shared_weight = 1; NULL = ones / zeros
 *   activation              gdn_activation_t
 * Limits: D % groups == 0, D / groups at most 8192, D at most 2^28, B T at most
 * 2^31 - 2^20 - 256.  Arithmetic in
 * float32, the mean taken off before squares are summed; one rounding at the end.
 * SiLU and the sigmoid come from the hardware's fast exponential and reciprocal, as in
 * short_conv_fwd.  An Inf or NaN in x stays within its token's group.
 */
typedef enum gdn_activation {
  GDN_ACT_NONE = 0,     /* v             */
  GDN_ACT_SILU = 1,     /* v / (1 + e^-v) */
  GDN_ACT_SIGMOID = 2   /* 1 / (1 + e^-v) */
} gdn_activation_t;

typedef struct group_norm_args {
  int32_t dtype;               /* gdn_dtype_t of x, z, y */
  int32_t weight_dtype;        /* gdn_dtype_t of weight, bias */
  const void *x, *z;
  const void *weight, *bias;
  void *y;
  int64_t x_stride, x_batch_stride, z_stride, z_batch_stride, y_stride, y_batch_stride;
  int32_t B, T, D, groups;
  int32_t shared_weight;
  int32_t center, gate_first;
  int32_t activation;          /* gdn_activation_t */
  float eps;                   /* >= 0 */
} group_norm_args;

gdn_status_t group_norm_fwd(const group_norm_args *args, gdn_stream_t stream);

/*
 * Gradient of group_norm_fwd.  The statistics are formed again from x; nothing of the
 * forward call is kept.
 *   dy, x, z, dx, dz [B, T, D]   dtype    strided; dx and dz must not overlap an input;
 *                                         dz is given exactly when z is
 *   dweight, dbias               float32  shaped as weight and bias, NULL = not returned
 * The sums over tokens run in a fixed order (float32 partial sums in `workspace`, 16-byte
 * aligned, group_norm_bwd_workspace_size() bytes), so results do not change from run to
 * run.  The rest as group_norm_fwd.
 */
typedef struct group_norm_bwd_args {
  int32_t dtype;               /* gdn_dtype_t of dy, x, z, dx, dz */
  int32_t weight_dtype;        /* gdn_dtype_t of weight, bias */
  const void *dy, *x, *z;
  const void *weight, *bias;
  void *dx, *dz;
  float *dweight, *dbias;
  int64_t dy_stride, dy_batch_stride, x_stride, x_batch_stride, z_stride, z_batch_stride;
  int64_t dx_stride, dx_batch_stride, dz_stride, dz_batch_stride;
  int32_t B, T, D, groups;
  int32_t shared_weight;
  int32_t center, gate_first;
  int32_t activation;
  float eps;
  void *workspace;
  size_t workspace_bytes;
} group_norm_bwd_args;

/* Bytes of workspace group_norm_bwd needs (0 when neither dweight nor dbias is returned);
 * reads sizes, strides, dtype, the tensors' alignment and which of them are NULL. */
gdn_status_t group_norm_bwd_workspace_size(const group_norm_bwd_args *args, size_t *bytes);
gdn_status_t group_norm_bwd(const group_norm_bwd_args *args, gdn_stream_t stream);

/*
 * KDA for T = 1..4 new tokens per batch entry against pooled states, updated in place:
 * the recurrence of kda_chunk_fwd with the gates formed as gdn_decode forms them, one per
 * key channel.  Per token, with S [V, K] of the entry's slot:
 *     decay[c] = exp(-e^A_log softplus(a[c] + dt_bias[c])),   beta = sigmoid(b)
 *     S <- S diag(decay),  d = beta (v - S k),  S <- S + d k^T,  o = scale S q
 * with softplus(x) = log(1 + e^x), x itself above 20.
 *   q, k     [B, T, H, K]   dtype    value head hv reads key head hv / (HV / H); divided
 *                                    by sqrt(sum x^2 + eps) when use_qk_l2norm
 *   v, o     [B, T, HV, V]  dtype    o float32 when o_fp32 = 1
 *   a        [B, T, HV, K]  dtype
 *   b        [B, T, HV]     dtype
 *   A_log    [HV], dt_bias [HV, K]  float32, dt_bias NULL = zeros
 *   state    [pool, HV, V, K]  state_dtype   K fastest; read once, carried over the T tokens
 *                                    in float32 and written once
 *   slot_indices [B]        int32    as gdn_decode
 * Token tensors are strided as in ssm_chunk_fwd: column ranges of wider buffers, so that q,
 * k and v may be columns of the short convolution's output.  Outputs must not overlap inputs.
 * A call that ends with GDN_ERR_TIMEOUT in the device error word leaves every row of the states
 * as the call's, or as it was.
 * Limits: 8 <= K <= 256, K % 8 == 0, HV % H == 0, HV at most 65535.  scale <= 0 selects
 * 1/sqrt(K); eps < 0 selects 1e-6.
 */
typedef struct kda_decode_args {
  int32_t dtype;               /* gdn_dtype_t of q, k, v, a, b, o */
  int32_t state_dtype;         /* gdn_dtype_t of state */
  const void *q, *k, *v, *a, *b;
  const float *A_log, *dt_bias;
  void *state;
  const int32_t *slot_indices;
  void *o;
  int64_t q_stride, q_batch_stride, k_stride, k_batch_stride, v_stride, v_batch_stride;
  int64_t a_stride, a_batch_stride, b_stride, b_batch_stride, o_stride, o_batch_stride;
  int32_t B, T, H, HV, K, V, pool;
  int32_t use_qk_l2norm;
  int32_t o_fp32;
  float scale, eps;
} kda_decode_args;

gdn_status_t kda_decode(const kda_decode_args *args, gdn_stream_t stream);

/*
 * GDN chunked forward without a workspace, for callers that cannot allocate
 * device memory (a host runtime that owns a fixed device-memory budget and
 * forbids cudaMalloc from plugins, or a latency-critical loop that must not
 * hit cudaMalloc's implicit synchronisation).  The pages have no counterpart
 * to this entry point; it is a convenience of this library.
 * Same arguments and results as gdn_chunk_fwd; `workspace` and
 * `workspace_bytes` are ignored.  Scratch comes from a fixed device array of
 * gdn_noalloc_scratch_bytes() bytes (32 MiB) that every GPU loading the
 * library holds until the process exits; a problem whose
 * gdn_chunk_workspace_size exceeds it returns GDN_ERR_WORKSPACE and enqueues
 * nothing.  All calls on a device share that array: calls that may overlap
 * on the GPU (e.g. on different streams) race and must be ordered by the
 * caller.  The first call on each device resolves the array's device address
 * (with that device current), so make it before any stream capture.
 */
gdn_status_t gdn_chunk_fwd_noalloc(const gdn_chunk_args *args, gdn_stream_t stream);

/* Size in bytes of the fixed scratch array used by gdn_chunk_fwd_noalloc. */
size_t gdn_noalloc_scratch_bytes(void);

/*
 * Self-test of the failure path shared by every kernel that waits on an
 * asynchronous copy or tensor-core operation: each such wait polls an
 * mbarrier a bounded number of times and, if the phase has not completed by
 * then, records GDN_ERR_TIMEOUT in the device error word and lets the kernel
 * finish instead of hanging.  This call runs that same wait once, in a
 * one-thread kernel, on a barrier of its own: with arrive = 0 nothing ever
 * arrives, so the wait gives up after max_polls polls (1 .. 2^22; the kernels
 * use 2^22) and GDN_ERR_TIMEOUT is recorded; with arrive = 1 the kernel
 * completes the phase itself first and nothing is recorded.  No copy or
 * tensor-core operation is in flight, so giving up leaves nothing behind.
 * Read the outcome with gdn_check_device_error().  GDN_ERR_INVALID_ARG for
 * arguments outside those ranges.
 */
gdn_status_t gdn_self_test_wait(int32_t arrive, int32_t max_polls, gdn_stream_t stream);

/*
 * Self-test of the bounds checks of a checked build (the library compiled
 * with -DGDN_CHECKED; the release build compiles them away).  Before a CTA of
 * any kernel touches memory, a checked build compares the index ranges the
 * CTA derived (chunk slots, token rows, heads, value columns, state slots)
 * with the extents of the tensors they index; when one falls outside, the CTA
 * records GDN_ERR_BOUNDS in the device error word and returns, uniformly and
 * before any barrier, so that nothing waits on it.  This call runs that check
 * in a one-CTA kernel on the index `index` against the extent `extent`: a
 * checked build records GDN_ERR_BOUNDS unless 0 <= index < extent, a release
 * build never does.  Read the outcome with gdn_check_device_error();
 * *checked_build is set to 1 in a checked build, else 0 (it may be NULL).
 */
gdn_status_t gdn_self_test_bounds(int32_t index, int32_t extent, int32_t *checked_build,
                                  gdn_stream_t stream);

/* Wait for `stream`, then read and clear the device error word of the current
 * device into *code (a gdn_status_t value, GDN_OK if nothing was recorded).
 * The word is shared by every stream of the device: the first error recorded
 * since the last clear is kept. */
gdn_status_t gdn_check_device_error(gdn_stream_t stream, int32_t *code);

/* Static, NUL-terminated name of a status. */
const char *gdn_status_string(gdn_status_t status);

/* Description of the calling thread's last host-side failure ("" if none). */
const char *gdn_last_error_message(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_GB300_H */
