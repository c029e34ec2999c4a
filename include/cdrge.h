/*
 * cdrge.h - C ABI of the MI355X (gfx950) CD-RGE hot path.
 *
 * One CD-RGE update step, as described for arXiv 2505.17852 ("Scaling Recurrent Neural Networks
 * to a Billion Parameters with Zero-Order Optimization"):
 *
 *   losses:  L(theta + eps p_i), L(theta - eps p_i) for K Rademacher probes p_i, each the mean
 *            next-token cross-entropy of a full LSTM forward pass (pith.science review, "What
 *            carries the argument": only scalar losses return; alex-wiki source note, "Method":
 *            complete recurrent forwards at perturbed weights, no differentiation through time);
 *   update:  theta <- theta - eta / (2 K eps) * sum_i (L(theta + eps p_i) - L(theta - eps p_i)) p_i
 *            (the review's update is the eta = eps case of the alex-wiki g-hat form), with every
 *            p_i regenerated from its seed (alex-wiki "Method": reconstructible random seeds).
 *
 * The split between cdrge_probe_losses and cdrge_update follows the pages' distributed scheme
 * (review, "What carries the argument": workers compute perturbed losses and return only scalar
 * losses; the update needs only those scalars and the seeds).
 *
 * Model (the pages say only "LSTM", next-character prediction): embedding Emb[V][E] -> n_layers
 * LSTM layers (gate rows i, f, g, o; one bias per layer; zero initial state) -> W_out[V][H] +
 * b_out[V] -> softmax cross-entropy of token t+1 given tokens 0..t. Loss = mean over B*T.
 * Flat parameter layout, tensor ids in order: 0 Emb[V][E]; per layer l: 1+3l W_ih[4H][in_l]
 * (in_0 = E, in_l = H), 2+3l W_hh[4H][H], 3+3l b[4H]; 1+3L W_out[V][H]; 2+3L b_out[V];
 * row-major, concatenated.
 *
 * Probe signs: seed_i = Philox4x32-10(key = base_seed, counter = (i, lo32(step), hi32(step), 1)),
 * words 0 | 1 << 32. Element (tensor t, row r, column c) of p_i: word (c >> 5) & 3, bit
 * ((c & 31) >> 1) | ((c & 1) << 4) of Philox4x32-10(key = seed_i, counter = (c >> 7, r, t, 0));
 * a set bit is -1, a clear bit +1.
 *
 * Precision. dtype F32: parameters, arithmetic and losses in float32. dtype BF16: parameters
 * stored as bf16; a perturbed weight is bf16(float(w) +- eps) rounded to nearest even; matrix
 * products take bf16 operands (activations are rounded to bf16 where they enter a product) and
 * accumulate in float32; cell state, gates, logits and losses are float32; the update adds in
 * float32 and rounds to bf16. dtype BF16_EXACT: as BF16, but the probe is added exactly (below).
 *
 * Conventions shared by every call:
 *   - Pointers named as device pointers must be device memory of the GPU that was current at
 *     cdrge_init; the caller owns them (the library never allocates or frees device memory).
 *   - Work is enqueued on the stream given to cdrge_init (a hipStream_t passed as void*; NULL is
 *     the default stream) and calls return after enqueueing. Only cdrge_sync_status waits.
 *   - Argument errors are reported synchronously and enqueue nothing. A failed launch returns
 *     CDRGE_ERR_DEVICE. A context is bound to one stream and is not thread-safe.
 */
#ifndef CDRGE_H
#define CDRGE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define CDRGE_ABI_VERSION 1u

typedef struct cdrge_ctx cdrge_ctx; /* opaque, host memory, owned by the library */

typedef enum {
  CDRGE_OK = 0,
  CDRGE_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, wrong abi_version, ... */
  CDRGE_ERR_UNSUPPORTED = 2, /* valid configuration that the kernels do not tile */
  CDRGE_ERR_WORKSPACE = 3,   /* workspace missing, too small or misaligned */
  CDRGE_ERR_DEVICE = 4,      /* a HIP runtime call or kernel launch failed */
  CDRGE_ERR_NONFINITE = 5    /* a probe loss was NaN or infinite; the update left theta as is */
} cdrge_status;

/* CDRGE_BF16_EXACT: bf16 parameters with the probe added exactly. A radius eps below the bf16
 * spacing of a weight (eps = 1e-4 against |w| around 2^-6 .. 2^-5) is swallowed when the perturbed
 * weight is rounded back to bf16; here every matrix product takes the stored weights W and the
 * exact bf16 operand eps' P, eps' = bf16(eps), into the same float32 accumulator:
 * (W +- eps' P) x = W x +- eps' (P x), twice the matrix-core work of CDRGE_BF16. Biases get
 * +- eps' p in float32; the perturbed embedding rows are rounded to bf16 (they are the first
 * product's activations); activations are rounded as for CDRGE_BF16. The update uses
 * eta / (2 K eps'), the radius actually applied. (alex-wiki source note, "Method": weights
 * perturbed by eps u_i; the pages fix no precision.) */
typedef enum { CDRGE_F32 = 0, CDRGE_BF16 = 1, CDRGE_BF16_EXACT = 2 } cdrge_dtype;

typedef struct {
  uint32_t abi_version;     /* must be CDRGE_ABI_VERSION */
  int32_t n_layers;         /* L >= 1 */
  int32_t vocab;            /* V */
  int32_t embed;            /* E */
  int32_t hidden;           /* H */
  int32_t batch;            /* B sequences per forward */
  int32_t seq_len;          /* T predicted positions; tokens are [B][T+1] */
  int32_t n_probes;         /* K probe pairs: 2K forwards per step */
  int32_t probes_per_chunk; /* probe pairs evaluated together; 0 = all K. Results do not depend on it */
  int32_t dtype;            /* cdrge_dtype */
  float eps;                /* probe radius */
  float lr;                 /* eta; the pages' runs use eta = eps */
  uint64_t base_seed;       /* root of the probe seed stream */
} cdrge_config;

/* Number of parameters d in the flat layout above, or -1 for an invalid configuration. */
int64_t cdrge_param_count(const cdrge_config* cfg);

/* CDRGE_OK if the configuration is valid and supported; otherwise the reason.
 * Supported: n_probes <= 1024, and
 *   F32 with n_layers <= 8 and E, H, V <= 65536 when the on-chip state of one workgroup - h and c
 *   of every layer, the gate pre-activations, the layer input and its tables of signed partial
 *   sums for up to 2 probe pairs x 8 sequences - fits in 128 KB (about
 *   4 * m * (2 L H + 5 max(E, H) + 4 H) bytes for m = 2 * pairs * sequences per workgroup, plus
 *   8 L H bytes of biases);
 *   BF16 and BF16_EXACT when E % 32 == 0, H % 32 == 0, V <= 64, and one probe chunk's activations stay within
 *   32-bit element offsets: (2 * probes_per_chunk * B + 256) * max(E, H) < 2^31 and
 *   4 H max(E, H) < 2^31. */
cdrge_status cdrge_check_config(const cdrge_config* cfg);

/* Device workspace, in bytes, that cdrge_init needs for this configuration (256-byte aligned
 * base required). It holds the probe seeds, per-step perturbation tables and the recurrent state
 * of one probe chunk; its size grows with probes_per_chunk. */
cdrge_status cdrge_workspace_bytes(const cdrge_config* cfg, size_t* bytes_out);

/* The K probe seeds of update step `step`, computed on the host into seeds_host[K]. */
cdrge_status cdrge_probe_seeds(const cdrge_config* cfg, uint64_t step, uint64_t* seeds_host);

/* Creates a context. params: device pointer to the d parameters (float32 or bf16 bit patterns,
 * per dtype), updated in place by cdrge_update. workspace: device pointer of at least
 * cdrge_workspace_bytes. stream: hipStream_t. Both buffers must outlive the context. */
cdrge_status cdrge_init(cdrge_ctx** ctx_out, const cdrge_config* cfg, void* params,
                        void* workspace, size_t workspace_bytes, void* stream);

/* Enqueues the 2K perturbed forward passes of step `step`.
 *   tokens: device int32 [B][T+1]; every entry must lie in [0, V) (checked on the device:
 *     an out-of-range token makes the step's losses NaN).
 *   losses: device float32 [2K]; losses[2i] = L(theta + eps p_i), losses[2i+1] = L(theta - eps p_i).
 *   seq_losses: device float32 [2K][B] or NULL; per-sequence sums over t of the cross-entropy.
 * theta is read only. */
cdrge_status cdrge_probe_losses(cdrge_ctx* ctx, const int32_t* tokens, uint64_t step,
                                float* losses, float* seq_losses);

/* Enqueues the update of step `step` from device losses[2K] (layout as above). If any loss is
 * not finite, theta is left unchanged and the next cdrge_sync_status reports
 * CDRGE_ERR_NONFINITE. */
cdrge_status cdrge_update(cdrge_ctx* ctx, uint64_t step, const float* losses);

/* cdrge_probe_losses followed by cdrge_update on the same stream. */
cdrge_status cdrge_step(cdrge_ctx* ctx, const int32_t* tokens, uint64_t step, float* losses);

/* Transduction form of cdrge_probe_losses, for the synthetic sequence-to-sequence tasks the pages
 * also train on (alex-wiki source note, "Evidence And Limits": copy, reverse and rolling sum,
 * where only the output part of a sequence is scored).
 *   inputs: device int32 [B][T], every entry in [0, V): the token fed at (b, t).
 *   targets: device int32 [B][T]: the token to predict at (b, t), in [0, V), or below zero for a
 *     position that is not scored.
 * The loss of a perturbed model is the mean cross-entropy over the scored positions of the batch
 * (NaN when none is scored or an entry is out of range); seq_losses, when not NULL, gets the
 * per-sequence sums over the scored positions. cdrge_probe_losses(tokens) is this call with
 * inputs = tokens[:, 0:T] and targets = tokens[:, 1:T+1]. */
cdrge_status cdrge_probe_losses_io(cdrge_ctx* ctx, const int32_t* inputs, const int32_t* targets,
                                   uint64_t step, float* losses, float* seq_losses);

/* cdrge_probe_losses_io followed by cdrge_update on the same stream. */
cdrge_status cdrge_step_io(cdrge_ctx* ctx, const int32_t* inputs, const int32_t* targets, uint64_t step,
                           float* losses);

/* Waits for the context's stream and reports deferred errors (non-finite losses, device
 * faults). Clears the non-finite flag. */
cdrge_status cdrge_sync_status(cdrge_ctx* ctx);

/* Releases the context (host memory only). */
void cdrge_destroy(cdrge_ctx* ctx);

/* Static, human-readable name of a status. */
const char* cdrge_status_string(cdrge_status status);

/* Text of the last HIP failure behind a CDRGE_ERR_DEVICE returned to the calling thread
 * ("" if none). The pointer stays valid until the thread's next failing call. */
const char* cdrge_last_error_detail(void);

/* Diagnostics: when enabled, every launch is bracketed by HIP events on the context's stream
 * and its duration is added to a per-kind total. kind: 0 recurrent gate kernel, 1 logits and
 * cross-entropy, 2 update, 3 per-step preparation and loss reduction. The events are timing-only
 * (created without a system-scope fence), so recording them adds no cache write-back between
 * kernels; they order nothing for other streams or the host. */
cdrge_status cdrge_set_timing(cdrge_ctx* ctx, int enable);

/* Total milliseconds and launch count per kind since the last reset (waits for the stream). */
cdrge_status cdrge_get_timing(cdrge_ctx* ctx, int kind, double* total_ms, int64_t* launches,
                              int reset);

/* Algorithmic work of the launches counted under `kind` so far: matrix-core flops for kinds 0
 * and 1 (2 * M * N * K of each product actually executed), bytes of parameters read and written
 * for kind 2. */
cdrge_status cdrge_get_work(cdrge_ctx* ctx, int kind, double* work);

/* Name of the kernel whose launches are timed under `kind` for this context's configuration
 * (kind 0: k_lstm_gates_bf16, k_lstm_f32 or k_lstm_f32_sliced; 1: k_logits_ce_bf16,
 * k_ce_f32_sliced, or "" when the persistent fp32 kernel computes the loss itself; 2: the update
 * kernel; 3 and invalid arguments: ""). Static storage, never freed. */
const char* cdrge_timed_kernel(const cdrge_ctx* ctx, int kind);

/* For callers that cannot allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid allocation): one whole step, as cdrge_step, with no context and no
 * caller workspace. The workspace lives in a static device array of the library, one per device
 * (held from library load until the process ends), of cdrge_noalloc_max_workspace_bytes()
 * bytes (64 MiB): configurations whose cdrge_workspace_bytes exceed it are rejected with
 * CDRGE_ERR_WORKSPACE before anything is enqueued (smaller probes_per_chunk shrinks the need).
 * The call allocates nothing: no hipMalloc, no hipFree, no library allocation of device memory.
 * params, tokens and losses are as for cdrge_init, cdrge_probe_losses and cdrge_step; stream is a
 * hipStream_t (NULL: the default stream). Every call on one device shares that device's array and
 * finds it as the previous call left it (the status words are cleared at the start of each call),
 * so calls that overlap on one device - on two streams, or from two threads - race and must be
 * ordered by the caller. A non-finite loss leaves theta unchanged; with no context, the caller
 * reads that from the losses it gets back. */
cdrge_status cdrge_step_noalloc(const cdrge_config* cfg, void* params, const int32_t* tokens,
                                uint64_t step, float* losses, void* stream);

/* Size in bytes of the static per-device scratch cdrge_step_noalloc uses. */
size_t cdrge_noalloc_max_workspace_bytes(void);

/* ============================================================================================
 * Operators of a population of language models.
 *
 * A step of the path above evaluates many models that share their weights. The calls below give
 * the same evaluation to models that differ by a low-rank term instead of a full sign probe, that
 * recur through a state space instead of an LSTM cell, and that learn from a teacher instead of
 * the next token: a projection shared by all rows with a low-rank adapter by row, a selective
 * scan with its short causal convolution, and a distillation loss with its mean by model. They
 * compose with each other; the calls above do not take their results: cdrge_update moves an LSTM's
 * tensors along full sign probes that it draws from seeds, of which losses of other models say
 * nothing.
 *
 * They need no context. Every call enqueues on `stream` (a hipStream_t; NULL is the default
 * stream) and returns; pointers are device memory of the current device, which must be the
 * stream's. Nothing is allocated, no call waits, and every call may be captured into a graph.
 * dtype is CDRGE_F32 or CDRGE_BF16 and types the tensors written below as `T`; strides count
 * elements between consecutive rows, whose own elements are adjacent. Sums, running maxima,
 * decays and states are float32 or wider; results are rounded to T once, to nearest even.
 * Inputs and outputs must not overlap unless a call says so. Index arrays are read on the
 * device: an entry out of range never reads or writes out of bounds, its effect is stated below.
 * A workspace serves one call at a time: calls that may overlap (two streams, two graphs
 * replayed at once) need one each. Its contents need no preparation.
 * ============================================================================================ */

/* ---- Selective scan -------------------------------------------------------------------------
 * Per token, a row of xbc holds n_heads * head_dim inputs, then n_groups * state_dim entries B,
 * then as many entries C (`channels` in all); dt holds n_heads step sizes before their bias and
 * softplus. Head h belongs to group h / (n_heads / n_groups). With q the token's place in its
 * sequence (positions + index within the call), e = conv_width and sequences starting at zero (rows
 * of xbc before the first are zeros, so a weight that is not finite makes NaN of them):
 *
 *   u_q     = silu(conv_bias + sum_{j < e} conv_weight[:, j] xbc_{q - e + 1 + j})     (x, B, C = u)
 *   step_q  = softplus(dt_q + dt_bias)                                               (by head)
 *   S_q     = exp(step_q decay) S_{q-1} + step_q x_q B_q^T                           [head_dim][state_dim]
 *   y_q     = S_q C_q + skip x_q, times silu(z_q) when z is given
 */
typedef struct {
  uint32_t abi_version; /* must be CDRGE_ABI_VERSION */
  int32_t dtype;        /* CDRGE_F32 or CDRGE_BF16 */
  int32_t n_heads;
  int32_t head_dim;     /* 1 .. 256 */
  int32_t n_groups;     /* divides n_heads */
  int32_t state_dim;    /* 1 .. 256 */
  int32_t conv_width;   /* 2 .. 4 */
} cdrge_scan_config;

typedef struct {
  const void* conv_weight; /* T [channels][conv_width], the last column meets the newest token */
  const void* conv_bias;   /* T [channels], or NULL */
  const float* decay;      /* [n_heads], negative for a state that fades */
  const float* skip;       /* [n_heads], or NULL */
  const float* dt_bias;    /* [n_heads], or NULL */
} cdrge_scan_weights;

/* Carried state. Slot s of a cache of n_slots holds one sequence's ring of the last conv_width
 * rows of xbc (row q at entry q mod conv_width) and its S of every head. conv_in and ssm_in are
 * read, conv_out and ssm_out written; an output may be its input's own pointer (update in place),
 * and otherwise gets the slot's whole contents, while slots that no sequence of the call names
 * are left as they are. All four are given, or none (every sequence starts at zero, nothing is
 * kept; slots and positions must be NULL then). */
typedef struct {
  const void* xbc;          /* T [n_tokens][channels] */
  int64_t xbc_stride;
  const void* dt;           /* T [n_tokens][n_heads] */
  int64_t dt_stride;
  const void* z;            /* T [n_tokens][n_heads * head_dim], or NULL */
  int64_t z_stride;
  void* y;                  /* T [n_tokens][n_heads * head_dim] */
  int64_t y_stride;
  int64_t n_tokens;         /* 0 .. 2^30 */
  int32_t n_seqs;           /* 1 .. 2^20 */
  int32_t n_slots;
  const int32_t* offsets;   /* [n_seqs + 1]: sequence i has the rows offsets[i] .. offsets[i+1] - 1
                               (may be none); NULL: n_tokens / n_seqs rows each, exactly */
  const int32_t* slots;     /* [n_seqs]; NULL: sequence i has slot i */
  const int32_t* positions; /* [n_seqs]: tokens that the slot has seen before this call; zero (or
                               less) starts the sequence at zero whatever the slot holds */
  const void* conv_in;      /* T [n_slots][conv_width][channels] */
  void* conv_out;
  const float* ssm_in;      /* [n_slots][n_heads][head_dim][state_dim], 16-byte aligned where
                               state_dim is a multiple of 4 */
  float* ssm_out;
} cdrge_scan_io;

/* Workspace, in bytes, of cdrge_scan_prompt for n_tokens tokens in n_seqs sequences (256-byte
 * aligned base required). Equal sequences of at most 16 tokens without a state need none. */
cdrge_status cdrge_scan_workspace_bytes(const cdrge_scan_config* cfg, int64_t n_tokens, int32_t n_seqs,
                                        size_t* bytes_out);

/* Whole prompts, or continued ones. positions NULL: every sequence starts at zero. Rows of y
 * outside every sequence are left as they are. Offsets that fall or leave [0, n_tokens] are
 * clamped into a rising row. A sequence whose slot is negative keeps no state (and starts at
 * zero). One whose slot is n_slots or more, or is named by an earlier sequence of the call, gets
 * NaN rows and touches no state. A token that is not finite may spoil outputs of its own sequence
 * from up to 63 tokens before it; other sequences are not affected. Products are formed of entries
 * rounded to 22 bits, or to 2^-38 of the largest of their kind in a head's 64 tokens where that is
 * more: magnitudes of u or S past 2^100 are treated as infinite, and below 2^-100 as zero. */
cdrge_status cdrge_scan_prompt(const cdrge_scan_config* cfg, const cdrge_scan_weights* weights,
                               const cdrge_scan_io* io, void* workspace, size_t workspace_bytes, void* stream);

/* One token for each of n_seqs = n_tokens sequences (offsets must be NULL, the state and positions
 * given). A row with a negative slot is padding: its y row and every state are left as they are.
 * Slots out of range or named twice: as for cdrge_scan_prompt. */
cdrge_status cdrge_scan_step(const cdrge_scan_config* cfg, const cdrge_scan_weights* weights,
                             const cdrge_scan_io* io, void* stream);

/* ---- Low-rank adapters beside a shared projection --------------------------------------------
 *   y_r = weight x_r + bias + scale_r up_a (down_a x_r),   a = row_adapter[r], scale_r = row_scale[r]
 * The rows of one antithetic pair of low-rank probes name the same adapter with scales of either
 * sign; the rows of requests name their own. */
typedef struct {
  uint32_t abi_version; /* must be CDRGE_ABI_VERSION */
  int32_t dtype;        /* CDRGE_F32 or CDRGE_BF16 */
  int32_t in_features;  /* K, 1 .. 2^20 */
  int32_t out_features; /* O, 1 .. 2^20 */
  int32_t n_adapters;   /* A, 0 .. 2^20 */
  int32_t max_rank;     /* R, 1 .. 128 */
} cdrge_adapter_config;

typedef struct {
  const void* weight;   /* T [O][K] */
  int64_t weight_stride;
  const void* bias;     /* T [O], or NULL */
  const void* down;     /* T [A][R][K] */
  const void* up;       /* T [A][O][R] */
  const int32_t* ranks; /* [A]: the rank in use of each adapter (entries past it are not used,
                           whatever they hold; clamped into [0, R]), or NULL: R each */
} cdrge_adapter_weights;

/* Workspace, in bytes, of cdrge_adapter_project for n_rows rows (256-byte aligned base required). */
cdrge_status cdrge_adapter_workspace_bytes(const cdrge_adapter_config* cfg, int64_t n_rows, size_t* bytes_out);

/* x: T [n_rows][K]; row_adapter: int32 [n_rows], negative for no adapter, or NULL (no row has
 * one); row_scale: float32 [n_rows] or NULL (1); y: T [n_rows][O]. n_rows may be 0, up to 2^30. A row
 * whose adapter is A or more gets NaN. A row's result does not depend on what other rows' inputs
 * or adapters hold, nor on their order. In bf16 and from a few rows on, scale_r down_a x_r enters
 * its product with up_a rounded to 16 bits. */
cdrge_status cdrge_adapter_project(const cdrge_adapter_config* cfg, const cdrge_adapter_weights* weights,
                                   int64_t n_rows, const void* x, int64_t x_stride, const int32_t* row_adapter,
                                   const float* row_scale, void* y, int64_t y_stride, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* ---- Distillation from a teacher's top logits ------------------------------------------------
 * Row r has top_k teacher entries (id, logit); an entry with a negative id or a logit of minus
 * infinity is absent. With tau the temperature, p the softmax of the present entries' logits / tau
 * and q the softmax of the student's whole row / tau:
 *
 *   row_loss = tau^2 sum_j p_j (log p_j - log q_{id_j}),   d row_loss / d logit_v = tau (q_v - sum_{j: id_j = v} p_j)
 *
 * A row without a present entry is not scored: its loss and gradient are zero. An id of vocab or
 * more makes its row NaN. An id may come twice. losses[m] is the mean of the scored rows of model
 * m, which owns the rows m (n_rows / n_models) onwards (NaN if it has none). Sums run in a fixed
 * order. */
typedef struct {
  uint32_t abi_version; /* must be CDRGE_ABI_VERSION */
  int32_t dtype;        /* type T of the logits and their gradient */
  int32_t vocab;        /* 1 .. 2^24 */
  int32_t top_k;        /* 1 .. 1024 */
  int32_t n_models;     /* 1 .. 2^20; divides the number of rows */
  float temperature;    /* 2^-60 .. 2^60 */
} cdrge_distill_config;

/* logits: T [n_rows][vocab]; ids: int32 [n_rows][top_k]; teacher: float32 [n_rows][top_k];
 * row_losses: float32 [n_rows]; losses: float32 [n_models], or NULL. n_rows may be 0, up to 2^30. */
cdrge_status cdrge_distill_losses(const cdrge_distill_config* cfg, int64_t n_rows, const void* logits,
                                  int64_t logits_stride, const int32_t* ids, const float* teacher,
                                  float* row_losses, float* losses, void* stream);

/* The same losses, and dlogits[r] = row_grad[r] * d row_loss_r / d logits_r (row_grad: float32
 * [n_rows], or NULL: 1) in T. dlogits may be logits itself (same pointer and stride). A logit of
 * minus infinity has q = 0. */
cdrge_status cdrge_distill_grad(const cdrge_distill_config* cfg, int64_t n_rows, const void* logits,
                                int64_t logits_stride, const int32_t* ids, const float* teacher,
                                const float* row_grad, float* row_losses, float* losses, void* dlogits,
                                int64_t dlogits_stride, void* stream);

/* ---- Gated delta rule -----------------------------------------------------------------------
 * A recurrence beside the scan, with the same cache of slots. Per token and head, a row of v holds
 * value_dim entries, rows of q and k key_dim entries for each of n_groups groups (head h belongs to
 * group h / (n_heads / n_groups)), dt and beta one entry a head before their functions:
 *
 *   q' = q_scale q / sqrt(q.q + norm_eps),   k' = k / sqrt(k.k + norm_eps)
 *   a_t = exp(decay softplus(dt_t + dt_bias)),   b_t = 1 / (1 + exp(-beta_t))                 (by head)
 *   S_t = a_t S_{t-1} + b_t (v_t - a_t S_{t-1} k'_t) k'_t^T                            [value_dim][key_dim]
 *   y_t = S_t q'_t
 *
 * The squares of a row of q or k must sum to less than 2^127 (magnitudes up to 2^59 always do); a row
 * past that counts as not finite, and so do magnitudes past 2^100 of v, of the state or of its product
 * with a row of q (for y alone) or of k as it comes. Of v, of the state and of v over the length of its
 * row of k, what is below 2^-100 may lose bits. */
typedef struct {
  uint32_t abi_version; /* must be CDRGE_ABI_VERSION */
  int32_t dtype;        /* CDRGE_F32 or CDRGE_BF16 */
  int32_t n_heads;
  int32_t value_dim;    /* 1 .. 256 */
  int32_t n_groups;     /* divides n_heads */
  int32_t key_dim;      /* 1 .. 256 */
  float q_scale;        /* finite, magnitude up to 2^60; key_dim^-0.5 is usual */
  float norm_eps;       /* 2^-60 .. 1 */
} cdrge_delta_config;

typedef struct {
  const float* decay;   /* [n_heads], negative for a state that fades */
  const float* dt_bias; /* [n_heads], or NULL */
} cdrge_delta_weights;

/* state_in is read and state_out written; they may be the same pointer (update in place), and
 * otherwise state_out gets the slot's whole contents, while slots that no sequence of the call names
 * are left as they are. Both are given, or none (every sequence starts at zero, nothing is kept; slots
 * and positions must be NULL then). */
typedef struct {
  const void* q;            /* T [n_tokens][n_groups * key_dim] */
  int64_t q_stride;
  const void* k;            /* T [n_tokens][n_groups * key_dim] */
  int64_t k_stride;
  const void* v;            /* T [n_tokens][n_heads * value_dim] */
  int64_t v_stride;
  const void* dt;           /* T [n_tokens][n_heads] */
  int64_t dt_stride;
  const void* beta;         /* T [n_tokens][n_heads] */
  int64_t beta_stride;
  void* y;                  /* T [n_tokens][n_heads * value_dim] */
  int64_t y_stride;
  int64_t n_tokens;         /* 0 .. 2^30 */
  int32_t n_seqs;           /* 1 .. 2^20 */
  int32_t n_slots;
  const int32_t* offsets;   /* as in cdrge_scan_io */
  const int32_t* slots;     /* as in cdrge_scan_io */
  const int32_t* positions; /* [n_seqs]: zero (or less) starts the sequence at zero whatever the slot holds */
  const float* state_in;    /* [n_slots][n_heads][value_dim][key_dim], 16-byte aligned where key_dim is a
                               multiple of 4 */
  float* state_out;
} cdrge_delta_io;

/* Workspace, in bytes, of cdrge_delta_prompt for n_tokens tokens in n_seqs sequences (256-byte
 * aligned base required). */
cdrge_status cdrge_delta_workspace_bytes(const cdrge_delta_config* cfg, int64_t n_tokens, int32_t n_seqs,
                                         size_t* bytes_out);

/* Whole prompts, or continued ones. Offsets, slots that are negative, out of range or named twice, and
 * rows outside every sequence: as for cdrge_scan_prompt. A token that is not finite may spoil outputs of
 * its own sequence from up to 63 tokens before it; other sequences are not affected. Short sequences go
 * token by token, others in blocks, by the call's sizes: the sums, in float32, have another order then. */
cdrge_status cdrge_delta_prompt(const cdrge_delta_config* cfg, const cdrge_delta_weights* weights,
                                const cdrge_delta_io* io, void* workspace, size_t workspace_bytes, void* stream);

/* One token for each of n_seqs = n_tokens sequences (offsets must be NULL, the state and positions
 * given). A row with a negative slot is padding: its y row and every state are left as they are. */
cdrge_status cdrge_delta_step(const cdrge_delta_config* cfg, const cdrge_delta_weights* weights,
                              const cdrge_delta_io* io, void* stream);

/* ---- Scores of given tokens -----------------------------------------------------------------
 * With tau the temperature, p the softmax of a row's logits / tau and t its given token:
 *
 *   logprob = log p_t,   entropy = -sum_v p_v log p_v   (a v of p_v = 0 adds nothing)
 *   d logprob / d logit_v = ((v == t) - p_v) / tau,   d entropy / d logit_v = -p_v (log p_v + entropy) / tau
 *
 * and the top_k alternatives are the largest logits, in falling order, equal ones by their place.
 * A negative token is padding: its logprob is zero, the row's entropy and alternatives are as for any
 * other. A token of vocab or more makes its logprob NaN. A logit of minus infinity has p = 0 and is no
 * alternative: places that are left over have the id -1 and the logprob minus infinity, which a
 * distillation loss takes for absent. A row with a NaN, plus infinity, or nothing but minus infinity
 * has NaN for its token's logprob, its entropy and its alternatives' logprobs, and -1 for their ids. */
typedef struct {
  uint32_t abi_version; /* must be CDRGE_ABI_VERSION */
  int32_t dtype;        /* type T of the logits and their gradient */
  int32_t vocab;        /* 1 .. 2^24 */
  int32_t top_k;        /* 0 .. 1024, at most vocab */
  float temperature;    /* 2^-60 .. 2^60 */
} cdrge_score_config;

/* logits: T [n_rows][vocab]; tokens: int32 [n_rows], or NULL where logprobs is; logprobs, entropy:
 * float32 [n_rows], either may be NULL; top_ids: int32 [n_rows][top_k] and top_logprobs: float32
 * [n_rows][top_k], NULL where top_k is 0. n_rows may be 0, up to 2^30. */
cdrge_status cdrge_token_scores(const cdrge_score_config* cfg, int64_t n_rows, const void* logits,
                                int64_t logits_stride, const int32_t* tokens, float* logprobs, float* entropy,
                                int32_t* top_ids, float* top_logprobs, void* stream);

/* dlogits[r] = d_logprob[r] * d logprob_r / d logits_r + d_entropy[r] * d entropy_r / d logits_r in T.
 * d_logprob, d_entropy: float32 [n_rows], either may be NULL (0; tokens may be NULL where d_logprob
 * is); d_logprob counts as zero where the token is padding. Where both are zero the row's gradient is
 * zero whatever it holds; otherwise a row that has NaN above, or a token of vocab or more with a
 * d_logprob that is not zero, gives NaN. Factors past 2^100 times the temperature count as not finite.
 * dlogits may be logits itself (same pointer and stride). */
cdrge_status cdrge_token_scores_grad(const cdrge_score_config* cfg, int64_t n_rows, const void* logits,
                                     int64_t logits_stride, const int32_t* tokens, const float* d_logprob,
                                     const float* d_entropy, void* dlogits, int64_t dlogits_stride, void* stream);

/* ---- Weights in microscaled 4-bit floating point ----------------------------------------------
 * A row of `in_features` values is kept as blocks of 32 (the last may be short): for each a scale
 * byte e and 16 bytes of codes, two values to a byte, the first in its low half, zeros past the end.
 * A code is a sign (8) and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6; the value is 2^(e - 127) times that.
 * Quantisation takes e so that the block's largest magnitude is in [4, 8) 2^(e - 127), or e = 0 where
 * that is too small, and the nearest code, ties to the even one, magnitudes past 6 becoming 6. A block
 * with a NaN or an infinity has e = 255, which stands for NaN in all of it. (OCP Microscaling Formats,
 * MXFP4: E2M1 elements, E8M0 scales.) */
typedef struct {
  uint32_t abi_version; /* must be CDRGE_ABI_VERSION */
  int32_t dtype;        /* type T of rows that are not quantised: CDRGE_F32 or CDRGE_BF16 */
  int32_t in_features;  /* K, 1 .. 2^20 */
  int32_t out_features; /* O, 1 .. 2^20 (used by cdrge_mx_project alone, checked by every call) */
} cdrge_mx_config;

/* x: T [n_rows][K]; codes: uint8 [n_rows][16 * ceil(K / 32)], 16-byte aligned; scales: uint8 [n_rows]
 * [ceil(K / 32)]. n_rows may be 0, up to 2^30. */
cdrge_status cdrge_mx_quantize(const cdrge_mx_config* cfg, int64_t n_rows, const void* x, int64_t x_stride,
                               uint8_t* codes, uint8_t* scales, void* stream);

/* The values that codes and scales stand for (either type holds all that quantisation makes exactly;
 * e = 253 and 254 may stand for more than T holds, and become infinite). */
cdrge_status cdrge_mx_dequantize(const cdrge_mx_config* cfg, int64_t n_rows, const uint8_t* codes,
                                 const uint8_t* scales, void* x, int64_t x_stride, void* stream);

/* Workspace, in bytes, of cdrge_mx_project for n_rows rows (256-byte aligned base required); the
 * largest of the calls' serves all of them on a stream. */
cdrge_status cdrge_mx_workspace_bytes(const cdrge_mx_config* cfg, int64_t n_rows, size_t* bytes_out);

/* y_r = W Q(x_r) + bias, with W the values of w_codes and w_scales [O][K] and Q(x_r) those of the row
 * quantised as by cdrge_mx_quantize. bias: T [O], or NULL; y: T [n_rows][O]. Products of codes are
 * exact and summed in float32. A row with a NaN or an infinity gives NaN; other rows are not affected.
 * y must not overlap x. The workspace may be NULL where cdrge_mx_workspace_bytes says 0 (few rows). */
cdrge_status cdrge_mx_project(const cdrge_mx_config* cfg, const uint8_t* w_codes, const uint8_t* w_scales,
                              const void* bias, int64_t n_rows, const void* x, int64_t x_stride, void* y,
                              int64_t y_stride, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CDRGE_H */
