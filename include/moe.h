/*
 * moe.h - C ABI of the GB300 (sm_103a) MoE layer library (libmoe.so): token routing and
 * expert compute, forward and backward, on one GPU.
 *
 * The layer (pages cited by title and section):
 *   z   = x Wg^T (+ bg)                                   gate linear
 *   idx = top-k of z per token (ties -> lower expert id)  top-k selection
 *   w   = softmax(z[idx] / temperature) over the k        routing weights
 *   k = E is dense soft routing (the naive soft MoE of the Expert-Parallelism page, section
 *   2.2: every expert runs on every token): nothing is selected, slot j holds expert j and
 *   w = softmax(z / temperature) over all E.
 *     "Native MoE training system PithTrain", section 4.1 (PithTrainMoELayer.forward:
 *     gate, torch.topk, softmax over the selected values); "Expert Parallelism: Scaling
 *     Mixture-of-Experts Models", section 2.2 (softmax(gate(x)/temperature); hybrid top-8
 *     pre-selection with soft weights over the 8), section 5.5 (route in FP32).
 *   counts[e], balance_loss = mean_e (counts[e] - mean(counts))^2
 *     "PyTorch distributed MoE training", section 3.3 (balance_loss).
 *   capacity C = ceil(capacity_factor * T * k / E); assignment (t,j) -> e is kept iff
 *   fewer than C earlier tokens picked e
 *     PithTrain page, section 4.3 item 1 (capacity, overflow tokens dropped).
 *   Xp = x rows permuted into expert buckets (token order inside a bucket)
 *     Expert-Parallelism page, section 4.2 idea 2 (tokens written straight into
 *     per-expert bucket offsets; one-device form of the sparse dispatch).
 *   per expert e: A = Xp_e W1_e^T + b1_e, H = GELU(A) (erf form), Yp = H W2_e^T + b2_e
 *     PyTorch-MoE page, section 3.2 (Expert); PithTrain page, section 4.1 (expert_pool).
 *   y[t] = sum over kept slots j of w[t,j] Yp[row(t,j)]
 *     PithTrain page, section 4.1 (output[mask] += expert_output * routing_weight).
 *   backward of L = sum(y * dy) (+ aux_loss_weight * balance_loss, which has no gradient)
 *     PithTrain page, section 4.2 (loss.backward()); PyTorch-MoE page, section 4.3
 *     (aux_loss_weight = 0.01).
 *
 * Conventions (every entry point):
 * - Pointers named as device pointers must point to device memory of the current device;
 *   host pointers are only the moe_config_t. The caller owns every buffer; the library
 *   allocates no device memory and keeps no per-call state. Outputs are overwritten.
 * - Activation, weight and scratch arrays (x, Wg, W1, b1, W2, b2, Xp, Gp, H, Yp, y, dy, dx,
 *   dW1, dW2 and ws) are read and written in 16-byte vectors and by TMA: their base
 *   addresses must be 16-byte aligned (cudaMalloc and PyTorch allocations are), else the
 *   call returns MOE_ERR_INVALID_ARG.
 * - All layouts are row-major, dense, following nn.Linear: x [T,d], Wg [E,d], bg [E] fp32,
 *   W1 [E,d_ff,d], b1 [E,d_ff], W2 [E,d,d_ff], b2 [E,d]. "act" below means the element
 *   type selected by cfg->dtype: fp32 (MOE_F32) or bf16 (MOE_BF16) for x, weights,
 *   activations and their gradients. Routing weights, logits and bias gradients are fp32.
 * - Permuted rows live in expert buckets: bucket e holds rows [offsets[e], offsets[e+1]),
 *   offsets[e] is a multiple of cfg->row_align (128 rows, set by moe_config_init), the
 *   first kept[e] rows are expert e's tokens in ascending token order and the rest of the
 *   bucket is padding (row_token = -1, zero rows in Xp). Buffers of permuted rows have
 *   cfg->rows_capacity rows.
 * - Calls are asynchronous on `stream` and never synchronise the host (except
 *   moe_get_error). Nothing that depends on data (counts, offsets) is read back.
 * - The library keeps a few per-device handles for the life of the process (its side stream,
 *   the device addresses of its error word and of the moe_dispatch_noalloc scratch array).
 *   cudaDeviceReset invalidates them: a process must not call the library on a device after
 *   resetting that device.
 * - Host-side validation failures return MOE_ERR_INVALID_ARG (bad value, null pointer) or
 *   MOE_ERR_UNSUPPORTED (valid but not implemented) and launch nothing. A failed launch
 *   returns MOE_ERR_CUDA. Faults detected on the device (a bounded wait that ran out, an
 *   index out of range) set a device error word that moe_get_error reports.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; 0 is the legacy default stream. */
typedef struct CUstream_st* moe_stream_t;

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = -1,
    MOE_ERR_UNSUPPORTED = -2,
    MOE_ERR_CUDA = -3,
    MOE_ERR_DEVICE_TIMEOUT = -4,
    MOE_ERR_DEVICE_BOUNDS = -5
} moe_status_t;

typedef enum { MOE_F32 = 0, MOE_BF16 = 1 } moe_dtype_t;

#define MOE_ROW_ALIGN 128   /* bucket alignment (rows); cfg->row_align */
#define MOE_MAX_EXPERTS 256
#define MOE_MAX_K 8           /* largest top-k selection; k = E (dense) is allowed for any E */

typedef struct {
    /* set by the caller */
    int32_t T;                 /* tokens, >= 0 */
    int32_t d;                 /* model dim, >= 1 */
    int32_t E;                 /* experts, 1..MOE_MAX_EXPERTS */
    int32_t k;                 /* experts per token: 1..min(E, MOE_MAX_K) (top-k), or E
                                  (dense soft routing, slot j = expert j) */
    int32_t d_ff;              /* expert hidden dim, >= 1 */
    float capacity_factor;     /* <= 0: no capacity limit */
    float temperature;         /* > 0: softmax(z_sel / temperature) */
    float aux_loss_weight;     /* weight of balance_loss in the reported loss (0.01 on the pages) */
    int32_t has_gate_bias;     /* 0/1: bg is added to the logits */
    int32_t dtype;             /* moe_dtype_t */
    float noise_std;           /* >= 0: training-time routing noise, logits += noise_std * N(0,1)
                                  before top-k and softmax ("PyTorch distributed MoE training",
                                  section 4.3: randn_like(logits) * 0.1); 0 = off */
    uint32_t noise_seed;       /* noise of experts 4g .. 4g+3 of token t: one Philox4x64-10
                                  draw at counter (t, g, 0, 0), key (noise_seed, 0); the top
                                  24 bits of outputs (0, 1) and (2, 3) give two pairs u1, u2 in
                                  (0,1], each turned into sqrt(-2 ln u1) cos(2 pi u2) and
                                  sqrt(-2 ln u1) sin(2 pi u2), in that order.
                                  Vary the seed from step to step. */
    /* derived by moe_config_init */
    int32_t capacity;          /* ceil(capacity_factor*T*k/E) in double, or INT32_MAX */
    int32_t rows_capacity;     /* rows of every permuted buffer (Xp, A, H, Yp) */
    int32_t row_align;         /* bucket alignment: MOE_ROW_ALIGN (128 rows). When the average
                                  bucket can reach 1024 rows (min(T*k, E*C)/E >= 1024) the
                                  expert GEMMs run 256-row tiles on CTA pairs (the last tile of
                                  a bucket with an odd number of 128-row tiles computes a second
                                  half it does not store); otherwise 128-row tiles on one CTA */
} moe_config_t;

/* Validates the caller's fields and fills the derived ones. Must be called before any
 * other entry point. Errors: MOE_ERR_INVALID_ARG (out-of-range field), MOE_ERR_UNSUPPORTED
 * (T*k or rows_capacity*max(d,d_ff) beyond 2^31-1). */
MOE_API moe_status_t moe_config_init(moe_config_t* cfg);

/* Bytes of device scratch (`ws`) the entry points need for this configuration; one buffer
 * of this size serves every call. Returns 0 for an invalid cfg. Aligned to 256 bytes. */
MOE_API size_t moe_workspace_bytes(const moe_config_t* cfg);

/* Gate linear + top-k + softmax over the k + expert counts + balance loss.
 *   x [T,d] act, Wg [E,d] act, bg [E] fp32 (read iff cfg->has_gate_bias, else may be NULL)
 *   -> idx [T,k] int32 (slot j = j-th largest logit; with k = E, slot j = expert j),
 *      w [T,k] fp32 (rows sum to 1), counts [E] int32 (pre-capacity choices, sum = T*k;
 *      T each with k = E), balance_loss [1] fp32,
 *      logits [T,E] fp32 (nullable: the routing logits z = x Wg^T + bg + noise; needed by
 *      moe_soft_balance).
 * Logits are accumulated in fp32. All pointers are device pointers. `ws` (moe_workspace_bytes)
 * holds the routing noise when cfg->noise_std > 0 (drawn once per call, then added to the
 * logits); it may be NULL when there is no noise. */
MOE_API moe_status_t moe_route(const moe_config_t* cfg, const void* x, const void* Wg, const float* bg,
                       int32_t* idx, float* w, int32_t* counts, float* balance_loss,
                       float* logits, void* ws, moe_stream_t stream);

/* Capacity, stable counting sort into expert buckets and the gather of x.
 *   idx [T,k] int32, x [T,d] act
 *   -> kept [E] int32 (= min(counts, capacity)), offsets [E+1] int32 (bucket starts,
 *      multiples of cfg->row_align, offsets[E] = rows in use), row_token [rows_capacity]
 *      int32 (token of each row; -1 on padding; rows >= offsets[E] unspecified),
 *      slot_row [T,k] int32 (row of assignment (t,j), -1 if dropped), n_dropped [1] int32,
 *      Xp [rows_capacity, d] act (rows >= offsets[E] unspecified).
 * Priority for capacity is token order. idx entries must lie in [0,E) and differ within a
 * token; a violation sets MOE_ERR_DEVICE_BOUNDS on the device. With k = E every bucket holds
 * tokens 0..min(T,C)-1 in order and idx must be the identity (idx[t,j] = j; else
 * MOE_ERR_DEVICE_BOUNDS); no sort runs. */
MOE_API moe_status_t moe_dispatch(const moe_config_t* cfg, const int32_t* idx, const void* x,
                          int32_t* kept, int32_t* offsets, int32_t* row_token, int32_t* slot_row,
                          int32_t* n_dropped, void* Xp, void* ws, moe_stream_t stream);

/* moe_dispatch for callers that cannot allocate device memory. The pages have no
 * counterpart: this entry point exists for code that may not call cudaMalloc (it runs
 * inside a memory budget or a host framework that owns every allocation, or it is a plugin
 * given only its input and output buffers) and so cannot provide the `ws` scratch.
 * Same arguments, results and errors as moe_dispatch, minus `ws`: the sort scratch is a
 * fixed array of MOE_NOALLOC_SCRATCH_BYTES in the library's device memory, reserved on
 * every GPU that loads the library until the process exits. The call allocates nothing.
 * Limits: T <= MOE_NOALLOC_MAX_TOKENS and T*k <= MOE_NOALLOC_MAX_ASSIGNMENTS; larger
 * configurations return MOE_ERR_UNSUPPORTED (use moe_dispatch with a workspace). With
 * k = E (dense routing) no sort and no scratch are used and the limits do not apply.
 * Each call looks up the array's device address (a host lookup; the first one on a device
 * may load the library's device code, so make a first call before any stream capture, as
 * for every entry point). All calls share the one array: calls that
 * may overlap on the GPU (other streams, other host threads) race and must be serialised
 * by the caller. Nothing in the array needs to start at zero; each call writes what it
 * reads. */
#define MOE_NOALLOC_SCRATCH_BYTES (2u << 20)
#define MOE_NOALLOC_MAX_TOKENS 65536
#define MOE_NOALLOC_MAX_ASSIGNMENTS 262144
MOE_API moe_status_t moe_dispatch_noalloc(const moe_config_t* cfg, const int32_t* idx, const void* x,
                                          int32_t* kept, int32_t* offsets, int32_t* row_token,
                                          int32_t* slot_row, int32_t* n_dropped, void* Xp,
                                          moe_stream_t stream);

/* Per-expert FFN over the buckets: A = Xp W1_e^T + b1_e, H = GELU(A), Yp = H W2_e^T + b2_e.
 *   Xp [rows_capacity,d], offsets [E+1] (from moe_dispatch), W1 [E,d_ff,d], b1 [E,d_ff],
 *   W2 [E,d,d_ff], b2 [E,d] -> Gp, H [rows_capacity,d_ff], Yp [rows_capacity,d] (all act;
 *   rows >= offsets[E] untouched). Gp = GELU'(A) = Phi(A) + A phi(A) is what the backward
 *   needs of the pre-activation, saved in place of A itself. fp32 accumulation. */
MOE_API moe_status_t moe_expert_ffn(const moe_config_t* cfg, const void* Xp, const int32_t* offsets,
                            const void* W1, const void* b1, const void* W2, const void* b2,
                            void* Gp, void* H, void* Yp, void* ws, moe_stream_t stream);

/* Weighted combine back to token order: y[t] = sum_{j: slot_row[t,j] >= 0} w[t,j] Yp[slot_row[t,j]],
 * accumulated in fp32; a token whose slots were all dropped gets 0.  y [T,d] act. */
MOE_API moe_status_t moe_combine(const moe_config_t* cfg, const void* Yp, const int32_t* slot_row,
                         const float* w, void* y, moe_stream_t stream);

/* Backward of the layer for the gradient seed dy [T,d] act, from the forward's saved tensors.
 *   inputs : dy, x, Wg, idx, w, offsets, row_token, slot_row, Xp, Gp, H, Yp, W1, W2 (as above),
 *            balance_loss [1] (nullable; enters the reported loss only)
 *   outputs: dx [T,d] act, dWg [E,d] fp32, dW1 [E,d_ff,d] act, db1 [E,d_ff] fp32,
 *            dW2 [E,d,d_ff] act, db2 [E,d] fp32, dbg [E] fp32 (nullable: gate-bias
 *            gradient, written only when cfg->has_gate_bias), dw [T,k] fp32 (nullable:
 *            gradient of the routing weights),
 *            loss [1] fp32 (nullable: sum(y*dy) + aux_loss_weight*balance_loss).
 * Dropped assignments give dw = 0 but still enter their token's softmax Jacobian. Experts
 * with no kept rows get zero weight and bias gradients. Scratch comes from ws. Part of the
 * work runs on a side stream of the library that forks from and joins back into `stream`
 * (event waits, also valid while `stream` is being captured into a CUDA graph). */
MOE_API moe_status_t moe_backward(const moe_config_t* cfg, const void* dy, const void* x, const void* Wg,
                          const int32_t* idx, const float* w, const int32_t* offsets,
                          const int32_t* row_token, const int32_t* slot_row, const void* Xp,
                          const void* Gp, const void* H, const void* Yp, const void* W1,
                          const void* W2, const float* balance_loss,
                          void* dx, float* dWg, void* dW1, float* db1, void* dW2, float* db2,
                          float* dbg, float* dw, float* loss, void* ws, moe_stream_t stream);

/* Differentiable balance loss on the soft expert load. The integer counts of balance_loss
 * ("PyTorch distributed MoE training", section 3.3) have no gradient; here the same
 * squared-deviation form is applied to the soft load of the gate probabilities
 * ("Expert Parallelism: Scaling Mixture-of-Experts Models", sections 2.2-2.3):
 *   P_e = sum_t softmax(logits_t / temperature)_e,  loss = weight * mean_e (P_e - T/E)^2.
 *   logits [T,E] fp32 (from moe_route) -> P [E] fp32, loss [1] fp32. Fixed-order sums.
 * Scratch from ws (moe_workspace_bytes covers it). */
MOE_API moe_status_t moe_soft_balance(const moe_config_t* cfg, const float* logits, float weight,
                                      float* P, float* loss, void* ws, moe_stream_t stream);

/* Gradient of moe_soft_balance's loss, ADDED to the layer gradients:
 *   dz_te = p_te (g_e - sum_j p_tj g_j) / temperature, g_e = weight * 2 (P_e - T/E) / E,
 *   dx += dz Wg, dWg += dz^T x, dbg += sum_t dz (dbg nullable).
 *   logits [T,E], P [E] (from moe_soft_balance), x [T,d] act, Wg [E,d] act;
 *   dx [T,d] act, dWg [E,d] fp32, dbg [E] fp32 are read and updated in place. */
MOE_API moe_status_t moe_soft_balance_backward(const moe_config_t* cfg, const float* logits,
                                               const float* P, float weight, const void* x,
                                               const void* Wg, void* dx, float* dWg, float* dbg,
                                               void* ws, moe_stream_t stream);

/* The soft balance loss on a sliding window of batches: "Expert Parallelism: Scaling
 * Mixture-of-Experts Models", section 2.3 (the per-expert load is averaged over the last 100
 * batches before the balance loss is taken, because a single batch's load is too noisy).
 * The caller owns the window's state; the library keeps none:
 *   ring  [W, E] fp32 device: the soft loads of the last W batches (contents need no
 *         initialisation: only slots written by earlier calls are read)
 *   state [2] int32 device: state[0] = ring slot of the next batch, state[1] = batches in the
 *         window (0..W). Set both to 0 before the first call; a state out of range sets
 *         MOE_ERR_DEVICE_BOUNDS and the window restarts.
 * Each call computes this batch's soft load P_e = sum_t softmax(logits_t / temperature)_e
 * (as moe_soft_balance), stores it in slot state[0], and with n = min(state[1] + 1, W):
 *   Pbar [E] = mean of the n most recent soft loads (this batch included),
 *   loss [1] = weight * mean_e (Pbar_e - mean(Pbar))^2   (loss nullable),
 * then advances the state: state[0] = (state[0] + 1) mod W, state[1] = n.
 * W = 1 is moe_soft_balance. logits [T,E] fp32; P, Pbar [E] fp32 device; W in
 * 1..MOE_MAX_WINDOW; ring and state 4-byte aligned. Scratch from ws (moe_workspace_bytes).
 * Successive calls on one ring must be ordered on the GPU (one stream). */
#define MOE_MAX_WINDOW 4096
MOE_API moe_status_t moe_soft_balance_window(const moe_config_t* cfg, const float* logits, float weight,
                                             int32_t W, float* ring, int32_t* state, float* P, float* Pbar,
                                             float* loss, void* ws, moe_stream_t stream);

/* Gradient of moe_soft_balance_window's loss, ADDED to the layer gradients. The earlier
 * batches of the window are stored statistics, so the gradient reaches only this batch:
 *   g_e = weight * 2 (Pbar_e - mean(Pbar)) / (E n),  n = state[1],
 *   dz_te = p_te (g_e - sum_j p_tj g_j) / temperature,  dx += dz Wg, dWg += dz^T x,
 *   dbg += sum_t dz (dbg nullable).
 * Call it after the forward call of the same batch (which set state[1] = n) and before the
 * next one, with that call's Pbar and state. logits, x [T,d] act, Wg [E,d] act; dx, dWg, dbg
 * are read and updated in place. */
MOE_API moe_status_t moe_soft_balance_window_backward(const moe_config_t* cfg, const float* logits,
                                                      const float* Pbar, float weight, const int32_t* state,
                                                      const void* x, const void* Wg, void* dx, float* dWg,
                                                      float* dbg, void* ws, moe_stream_t stream);

/* Expert co-selection matrix of a batch: "Expert Parallelism: Scaling Mixture-of-Experts
 * Models", section 3.2, step 1 (experts chosen by the same token; the input of the page's
 * affinity-aware placement). The page calls the matrix asymmetric; accordingly, for i != j,
 *   H[i][j] = number of tokens whose top-k holds i in an earlier slot (higher logit) than j,
 * so H + H^T is the co-occurrence count, and H[i][i] = number of tokens that chose i.
 *   idx [T,k] int32 (as from moe_route) -> H [E,E] int32 (overwritten). Device pointers.
 * Entries out of [0,E) or repeated within a token set MOE_ERR_DEVICE_BOUNDS and are skipped.
 * With k = E > MOE_MAX_K (dense routing) idx must be the identity: H[i][j] = T for i <= j,
 * 0 below the diagonal; a token whose row is not the identity sets MOE_ERR_DEVICE_BOUNDS and
 * is not counted. */
MOE_API moe_status_t moe_coselect(const moe_config_t* cfg, const int32_t* idx, int32_t* H,
                                  moe_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * The layer in a training step: token embedding (the layer's x, and the gradient that takes
 * its dx), the policy loss on the logits, and the AdamW step over the weights. The pages train
 * the layer inside such a step (PithTrain page, section 4.1) and leave these parts to the host
 * framework. The conventions at the top of this file hold; each call has a small
 * configuration of its own, checked on every call (nothing to initialise). */

/* Token embedding. W [V,d] act, ids [T] int32.
 *   moe_embed:          y[t] = scale * W[ids[t]]                      (y [T,d] act, one rounding)
 *   moe_embed_backward: dW[v] = scale * sum over tokens t with ids[t] = v of dy[t]
 * dy [T,d] act, dW [V,d] in grad_dtype. accumulate = 0 writes all of dW (zero rows for tokens
 * that do not occur); accumulate = 1 adds to dW and touches only the rows of tokens that do
 * (a table tied to the output head). Tokens equal to padding_id get no gradient (-1: none);
 * the forward looks them up like any other. Sums are fp32 in a fixed order (tokens sorted
 * stably by id), so results repeat bit for bit. An id outside [0,V) sets
 * MOE_ERR_DEVICE_BOUNDS: its y row is zero and its dy row is left out.
 * W, y, dy, dW and ws are 16-byte aligned; T = 0 is allowed (an overwritten dW is zeroed). */
typedef struct {
    int32_t T;             /* tokens, 0 .. 2^31 - 4097 */
    int32_t V;             /* rows of the table, 1 .. 2^31 - 4097 */
    int32_t d;             /* row length, 1 .. 2^28 */
    float scale;           /* finite */
    int32_t padding_id;    /* in [-1, V) */
    int32_t dtype;         /* moe_dtype_t of W, y, dy */
    int32_t grad_dtype;    /* moe_dtype_t of dW */
    int32_t accumulate;    /* 0/1 */
} moe_embed_config_t;
MOE_API moe_status_t moe_embed(const moe_embed_config_t* cfg, const int32_t* ids, const void* W, void* y,
                               moe_stream_t stream);
/* Bytes of `ws` for moe_embed_backward; 0 for an invalid cfg. */
MOE_API size_t moe_embed_workspace_bytes(const moe_embed_config_t* cfg);
MOE_API moe_status_t moe_embed_backward(const moe_embed_config_t* cfg, const int32_t* ids, const void* dy,
                                        void* dW, void* ws, moe_stream_t stream);

/* Clipped policy loss with a KL term, on the logits of the chosen tokens.
 *   lp = log softmax(logits[t] / temperature)[target[t]],   r = exp(lp - old_logp[t]),
 *   u  = ref_logp[t] - lp,
 *   l  = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl_weight (exp(u) - u - 1),
 *   loss = sum_t weight[t] l_t          (A = advantage[t]; weight carries mask and mean)
 *   dlogits[t,v] = weight[t] / temperature * dl/dlp * (1[v = target[t]] - softmax_v),
 *   dl/dlp = (-A r where r A <= clip(r) A, else 0) + kl_weight (1 - exp(u)).
 * logits [T,V] act with rows ld elements apart; dlogits [T,V] act, rows ld_grad apart; it may be
 * logits itself (then ld_grad = ld), any other overlap is not allowed. target [T] int32;
 * advantage, old_logp, ref_logp, weight, logp [T] fp32; loss [1] fp32. One reading of the
 * logits gives the loss and the gradient.
 *   old_logp null: on-policy, r = 1 with its gradient. Where old_logp[t] is the lp that this call
 *   computes, bit for bit, r is exactly 1 too; otherwise lp enters r with more than its 24 bits.
 *   moe_token_logp gives those bits for the same logits, T, V, ld, dtype and temperature; with
 *   another T or ld a row may be added up in another order, and lp differs by its rounding.
 *   ref_logp: needed iff kl_weight != 0.
 *   weight null: 1 for each token. logp, loss, dlogits: each may be null (not wanted).
 *   ws (moe_policy_workspace_bytes): needed when loss is not null.
 * A token with weight 0 or a negative target is left out: its logits are not read, whatever
 * they hold, logp = 0 and its dlogits row is zero. A target >= V sets MOE_ERR_DEVICE_BOUNDS and
 * the token is left out. Logits of -inf are tokens of probability 0; a row whose every logit
 * is -inf, or that holds +inf or NaN, has no distribution and gives NaN (row and loss).
 * Softmax statistics and loss sums are fp32, in a fixed order. logits and dlogits start on a
 * 16-byte boundary; V, ld, ld_grad may be odd. */
typedef struct {
    int32_t T;             /* tokens, 0 .. 2^31 - 4097 */
    int32_t V;             /* vocabulary, 1 .. 2^30 */
    int64_t ld;            /* elements between logits rows, >= V */
    int64_t ld_grad;       /* elements between dlogits rows, >= V */
    int32_t dtype;         /* moe_dtype_t of logits and dlogits */
    float temperature;     /* > 0 */
    float clip_low;        /* in [0, 1] */
    float clip_high;       /* >= 0 */
    float kl_weight;       /* finite */
} moe_policy_config_t;
/* Bytes of `ws` for moe_policy_loss; 0 for an invalid cfg. */
MOE_API size_t moe_policy_workspace_bytes(const moe_policy_config_t* cfg);
MOE_API moe_status_t moe_policy_loss(const moe_policy_config_t* cfg, const void* logits, const int32_t* target,
                                     const float* advantage, const float* old_logp, const float* ref_logp,
                                     const float* weight, float* logp, float* loss, void* dlogits, void* ws,
                                     moe_stream_t stream);
/* lp alone (what old_logp and ref_logp are made of, and what a server returns beside a sampled
 * token): T, V, ld, dtype and temperature of cfg. A negative target gives logp = 0. */
MOE_API moe_status_t moe_token_logp(const moe_policy_config_t* cfg, const void* logits, const int32_t* target,
                                    float* logp, moe_stream_t stream);

/* AdamW over many tensors in one call. With t = steps done + 1, g = grad (times *grad_scale):
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2,
 *   x = x (1 - lr weight_decay) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps),
 * all in fp32. x is the fp32 master if there is one (p is then x rounded to its type), else p.
 * States: fp32 m and v [n]; or, where m_scale and v_scale are given, 8 bits each: m holds
 * e4m3 values of m, v holds e4m3 values of sqrt(v), both times one fp32 scale to a block of
 * MOE_ADAMW_BLOCK elements (m_scale, v_scale [ceil(n / MOE_ADAMW_BLOCK)]: the power of two that
 * leaves the block's largest magnitude in [128, 256), 0 for a block below 2^-100). They are
 * rounded up or down by a dither of element and step (cfg->rounding): rounding to nearest would
 * hold sqrt(v) still, because beta2 = 0.999 moves it by 0.05 % a step and half a step of e4m3 is
 * 3 to 6 %. sqrt(v) > 0 never becomes 0. A value that is not finite is held as NaN and
 * leaves the rest of its block alone. The step itself uses m and v before they are rounded.
 * Zeroed states (and scales) are the start of training. Arrays are 16-byte aligned (scales,
 * lr, grad_scale: 4), tensors do not overlap; n = 0 is allowed.
 *   cfg, tensors [count]: host memory, read before the call returns
 *   lr: device fp32, replaces cfg->lr (a schedule under a captured graph); null: cfg->lr
 *   grad_scale: device fp32, multiplies every gradient (clipping, unscaling); null: 1
 *   state: MOE_ADAMW_STATE_BYTES of device memory, 8-byte aligned: the steps done, advanced by
 *     the call; zeroed before the first. Layout: 1 - beta1^t and 1 - beta2^t (double), t (int64),
 *     and 8 bytes that are zero between calls. Calls on one state are ordered on the GPU. */
#define MOE_ADAMW_BLOCK 256
#define MOE_ADAMW_STATE_BYTES 32
/* How 8-bit states are rounded. With s the share of the way from the held value below to the one
 * above, and d 20 bits of dither, the upper one is taken where s + d / 2^20 >= 1.
 *   MOE_ADAMW_ROUND_EVEN: d from a hash of element and step, one for m and one for v; v's share is
 *     taken between the squares. m and v are right on average (beta2 = 0.999, simulated: v to 0.2 %
 *     on constant gradients, 1.7 % on random ones).
 *   MOE_ADAMW_ROUND_WEYL: d the top 20 bits of i 0x9E3779B1 + t 0x61C88647 (mod 2^32) for element i
 *     of a tensor in step t; for v with its top bit turned, and the share taken in sqrt(v) itself.
 *     Fewer instructions, but v comes out high where beta2 is near 1: by 5 to 6 % at 0.999, up to 2 at
 *     0.99, within 1 at 0.95 (4096 elements over 3000 steps, simulated). */
#define MOE_ADAMW_ROUND_EVEN 0
#define MOE_ADAMW_ROUND_WEYL 1
typedef struct {
    double lr, beta1, beta2, eps;   /* lr finite, betas in [0, 1), eps in [1e-30, 1e30] */
    int32_t rounding;               /* MOE_ADAMW_ROUND_*: 8-bit states only */
    int32_t reserved;               /* 0 */
} moe_adamw_config_t;
typedef struct {
    void* p;                /* [n] weights, dtype */
    const void* g;          /* [n] gradient, grad_dtype */
    float* master;          /* [n] fp32 weights, or null */
    void* m;                /* [n] fp32, or e4m3 when m_scale is set */
    void* v;                /* [n] fp32, or e4m3 of the root when v_scale is set */
    float* m_scale;         /* both or neither */
    float* v_scale;
    int64_t n;              /* elements, 0 .. 2^38 */
    int32_t dtype;          /* moe_dtype_t */
    int32_t grad_dtype;     /* moe_dtype_t */
    float weight_decay;     /* finite, >= 0 */
    int32_t reserved;       /* 0 */
} moe_adamw_tensor_t;
MOE_API moe_status_t moe_adamw(const moe_adamw_config_t* cfg, const moe_adamw_tensor_t* tensors, int32_t count,
                               const float* lr, const float* grad_scale, void* state, moe_stream_t stream);

/* Choice of experts from scores: what moe_route's top-k and softmax over the k do not cover. The
 * scores are a softmax over all experts or sigmoids; a bias for balance enters the choice but not
 * the weights; experts may stand in groups, of which only the best are open to a token. Scores are
 * compared as hardware exponentials and reciprocals give them: within 2^-21 of the exact score for a sigmoid,
 * 2^-19 for a softmax (E = 256; absolute bounds: scores far below 1 may round alike), plus the rounding of
 * score + bias and, for groups, of the sum of two. Weights are rounded as fp32 operations are.
 *   logits [T,E] fp32 (moe_route's `logits`), bias [E] fp32 (nullable: 0)
 *   s_te = softmax(logits_t / temperature)_e   or   1 / (1 + exp(-logits_te / temperature)),
 *   c_te = s_te + bias_e; -inf where the logit is -inf or c is NaN,
 *   worth of a group (E / groups adjacent experts): the largest c in it, or the sum of its two
 *     largest (group_top 2, one expert alone: its c); the groups_kept of most worth stay open,
 *   idx [T,k] int32: the k largest c of the open groups, in falling order,
 *   w [T,k] fp32: scale * s[idx]; renormalise: divided by the sum of the k chosen scores (softmax:
 *     the softmax over the chosen logits alone; sigmoid: the sum plus 1e-20),
 *   counts [E] int32: choices of each expert (nullable), balance_loss [1] fp32 =
 *     mean_e (counts[e] - T k / E)^2 as moe_route's (nullable).
 * Ties, of experts and of groups, go to the lower id. Without a bias experts are compared by their logits
 * (and groups by the largest, with group_top 1), so that scores which round alike keep their order. idx are
 * always k different experts of the open groups; one with a logit of -inf is taken only where the
 * open groups hold fewer than k others, and has weight 0. A softmax over a row that holds NaN or
 * +inf is NaN: the row's weights are NaN and its experts the first ones. A row of -inf alone has
 * weights 0. logits are 16-byte aligned. ws (moe_route_scores_workspace_bytes) is needed when counts
 * or balance_loss is wanted. */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score_t;
typedef struct {
    int32_t T;             /* tokens, 0 .. 2^27 */
    int32_t E;             /* experts, 1 .. MOE_MAX_EXPERTS */
    int32_t k;             /* experts per token, 1 .. min(MOE_MAX_K, E / groups * groups_kept) */
    int32_t score;         /* moe_score_t */
    int32_t groups;        /* 1 .. 32, divides E; 1: no groups */
    int32_t groups_kept;   /* 1 .. groups */
    int32_t group_top;     /* 1 or 2 */
    int32_t renormalise;   /* 0/1 */
    float temperature;     /* > 0, finite; log2(e) / temperature too (temperature from 4.24e-39 on) */
    float scale;           /* finite */
} moe_score_config_t;
/* Bytes of `ws` for moe_route_scores on the current device (by its number of SMs); 0 for an invalid cfg. */
MOE_API size_t moe_route_scores_workspace_bytes(const moe_score_config_t* cfg);
MOE_API moe_status_t moe_route_scores(const moe_score_config_t* cfg, const float* logits, const float* bias,
                                      int32_t* idx, float* w, int32_t* counts, float* balance_loss, void* ws,
                                      moe_stream_t stream);
/* Gradient of sum(w * dw) in the logits, for the experts that were chosen (the choice itself and the
 * bias have none): dlogits [T,E] fp32, all of it written. Chosen scores alone have a gradient, but for
 * a softmax that is not renormalised, where every expert's does; only that one reads logits of experts
 * that were not chosen. An idx outside [0,E), or an expert that an earlier slot of the token holds, sets
 * MOE_ERR_DEVICE_BOUNDS and its slot is left out. A chosen logit of -inf has gradient 0 (a softmax over
 * -inf alone, too). logits and dlogits are 16-byte aligned and do not overlap. */
MOE_API moe_status_t moe_route_scores_backward(const moe_score_config_t* cfg, const float* logits,
                                               const int32_t* idx, const float* dw, float* dlogits,
                                               moe_stream_t stream);
/* moe_backward for a layer whose idx and w came from moe_route_scores: the same arguments and outputs,
 * with the gradient of the gate taken through the scores. scores->T, E and k are cfg's; logits [T,E] as
 * given to moe_route_scores; dlogits [T,E] fp32 is written as moe_route_scores_backward writes it, and
 * dx, dWg and dbg hold its part. cfg->temperature is not used. Dropped assignments give dw = 0 but still
 * enter their token's Jacobian. A softmax that is not renormalised has its part of dx (dlogits Wg) added to dx in the
 * layer's type: in bf16 dx is rounded twice, and off by up to a whole step of bf16. k = E is refused (MOE_ERR_UNSUPPORTED): dense routing wants slot j to be
 * expert j, and there is nothing to choose. */
MOE_API moe_status_t moe_backward_scores(const moe_config_t* cfg, const moe_score_config_t* scores,
                                         const float* logits, float* dlogits, const void* dy, const void* x,
                                         const void* Wg, const int32_t* idx, const float* w,
                                         const int32_t* offsets, const int32_t* row_token,
                                         const int32_t* slot_row, const void* Xp, const void* Gp, const void* H,
                                         const void* Yp, const void* W1, const void* W2,
                                         const float* balance_loss, void* dx, float* dWg, void* dW1, float* db1,
                                         void* dW2, float* db2, float* dbg, float* dw, float* loss, void* ws,
                                         moe_stream_t stream);

/* Layer norm of rows, and of a residual sum in the same pass.
 *   s = x + residual (residual null: s = x),  mean = mean(s),  rstd = 1 / sqrt(mean((s - mean)^2) + eps),
 *   y = (s - mean) rstd gain + bias                                   (gain null: 1; bias null: 0)
 * x, residual, y, total [T,d] act; gain, bias [d] in param_dtype; total = s, each element rounded once
 * (wanted iff residual is given); y is of the sum before it is rounded; mean, rstd [T] fp32 (each may be
 * null). y or total may be x or residual; any other overlap is not allowed. The mean is taken first, the
 * squares of the differences after it, in fp32 and a fixed order.
 * Backward, with g = dy gain and h = (s - mean) rstd:
 *   dx = rstd (g - mean(g) - h mean(g h)) + dtotal                     (dtotal null: 0)
 *   dgain = sum_t dy h,  dbias = sum_t dy      fp32 [d], each may be null; accumulate: added to them
 * s [T,d] act is the forward's total (or x), mean and rstd the forward's; dtotal [T,d] act is the gradient
 * that reaches the sum itself (a residual stream). dx may be dy, s or dtotal; any other overlap is not
 * allowed. dx may be null where only dgain or dbias is wanted. ws (moe_norm_workspace_bytes) is needed
 * with dgain or dbias; their sums are fp32 in a fixed order, so results repeat bit for bit.
 * T = 0 is allowed (dgain and dbias are zeroed unless accumulate). A row of s that holds NaN or an infinity
 * gives NaN in its own y and dx and in all of dgain, and leaves dbias, the sum of dy, alone. What is not finite in
 * dy leaves no finite element in its row of dx, and none in its column of dgain and dbias. Sums and squares are
 * fp32: a row whose sum passes it gives NaN, one whose sum of squares alone does has rstd = 0 and y = bias. Arrays of rows, gain, bias, dgain, dbias and ws are 16-byte aligned;
 * d may be odd. */
typedef struct {
    int32_t T;             /* rows, 0 .. 2^30 */
    int32_t d;             /* row length, 1 .. 2^20 */
    float eps;             /* finite, >= 0 */
    int32_t dtype;         /* moe_dtype_t of x, residual, y, total, dy, dx, dtotal */
    int32_t param_dtype;   /* moe_dtype_t of gain and bias */
    int32_t accumulate;    /* 0/1: backward adds to dgain and dbias */
} moe_norm_config_t;
MOE_API moe_status_t moe_layer_norm(const moe_norm_config_t* cfg, const void* x, const void* residual,
                                    const void* gain, const void* bias, void* total, void* y, float* mean,
                                    float* rstd, moe_stream_t stream);
/* Bytes of `ws` for moe_layer_norm_backward on the current device (by its number of SMs); 0 for an invalid cfg. */
MOE_API size_t moe_norm_workspace_bytes(const moe_norm_config_t* cfg);
MOE_API moe_status_t moe_layer_norm_backward(const moe_norm_config_t* cfg, const void* dy, const void* s,
                                             const void* gain, const float* mean, const float* rstd,
                                             const void* dtotal, void* dx, float* dgain, float* dbias, void* ws,
                                             moe_stream_t stream);

/* Orthogonalised updates of weight matrices (Muon), for a stack of `count` matrices [rows, cols], each on
 * its own (an MoE layer's W1 or W2: one matrix to an expert).
 *   orth(u): X = u / (|u| + eps) with |u| the root of the sum of squares; `steps` times, with A = X X^T
 *   (X^T X where rows > cols):  X = a X + (b A + c A A) X   (A on the right where rows > cols).
 * The singular values go near 1 and the directions stay; a matrix of zeros stays zero.
 *   moe_orthogonalize: o = orth(g)    o [count,rows,cols] in dtype, g in grad_dtype
 *   moe_muon:          m = momentum m + g (g times *grad_scale),  u = nesterov ? g + momentum m : m,
 *                      x = x (1 - lr weight_decay) - lr scale orth(u)
 * m [count,rows,cols] fp32 (zeroed before the first step); x is the fp32 master if there is one (p is then
 * x rounded to its type), else p in dtype. precision: MOE_BF16: operands of the products hold 11 bits (fp16,
 * scaled), X between the steps 22, sums are fp32; MOE_F32: operands hold two fp16 parts, 22 bits.
 * How far orth(u) is off, as a share of its size (root of the sums of squares; 5 steps, the usual
 * coefficients): MOE_BF16: about 1e-3, half of a rounding to bf16, at any rank of u: 2e-3 at most of what was
 * measured, 3e-3 of what was simulated (6e-3 with fewer than 16 rows or columns). MOE_F32: 1e-6 to 5e-6 at
 * full rank. Where u's rank is lower, roundings in the directions that it lacks grow by `a` with every step, as
 * they do in fp32 products: 2e-6 to 1.2e-5 at half to a quarter of it, 5e-5 at rank 1 (fp32 products: 1.4e-4). An element
 * that is not finite, or a matrix whose sum of squares is beyond fp32, gives NaN in all of its own matrix
 * and leaves the others alone.
 * lr (device fp32, replaces cfg->lr) and grad_scale (device fp32) may be null, as in moe_adamw. p, g, o,
 * master, m and ws (moe_muon_workspace_bytes) are 16-byte aligned and do not overlap, but o may be g where
 * their types are the same. count = 0 is allowed.
 * Coefficients and steps with which a singular value in [0, 1] can bring X or A = X X^T above 31.9, or b A + c A A
 * above 63.8 (all of them held in fp16, scaled), are refused (MOE_ERR_UNSUPPORTED); the usual ones stay below 1.5 and 3. */
typedef struct {
    int32_t count;         /* matrices, 0 .. 65535; count * ceil(rows / 256) * ceil(cols / 256) to 2^30 */
    int32_t rows, cols;    /* 1 .. 65536 each */
    int32_t steps;         /* 0 .. 100 */
    double a, b, c;        /* coefficients, magnitudes up to 16; see above */
    double lr, momentum, weight_decay, scale, eps;   /* finite; momentum in [0, 1), eps in [1e-12, 1] */
    int32_t nesterov;      /* 0/1 */
    int32_t dtype;         /* moe_dtype_t of p, o */
    int32_t grad_dtype;    /* moe_dtype_t of g */
    int32_t precision;     /* moe_dtype_t: how exact orth(u) is */
} moe_muon_config_t;
/* Bytes of `ws`; 0 for an invalid cfg or count = 0. */
MOE_API size_t moe_muon_workspace_bytes(const moe_muon_config_t* cfg);
MOE_API moe_status_t moe_orthogonalize(const moe_muon_config_t* cfg, const void* g, void* o, void* ws,
                                       moe_stream_t stream);
MOE_API moe_status_t moe_muon(const moe_muon_config_t* cfg, void* p, const void* g, float* master, float* m,
                              const float* lr, const float* grad_scale, void* ws, moe_stream_t stream);

/* Synchronises `stream`, then returns and clears the device error word of the current
 * device: MOE_OK, MOE_ERR_DEVICE_TIMEOUT or MOE_ERR_DEVICE_BOUNDS; MOE_ERR_CUDA if the
 * stream reports a CUDA error. */
MOE_API moe_status_t moe_get_error(moe_stream_t stream);

/* Self-test of the device-side bounded waits (failure detection without a GPU fault). A
 * kernel waits on an object that nothing signals, through the wait helper the layer's kernels
 * use: an mbarrier phase wait, as in the tensor-core pipelines (mode 0, the only mode). After
 * budget_cycles (1e3 .. 4e9 SM clock cycles) the wait gives up, records
 * MOE_ERR_DEVICE_TIMEOUT in the device error word and the kernel returns; the context stays
 * usable.
 *   timed_out: device int32, set to the number of waits that ran out (1)
 *   scratch  : unused (may be null)
 * Returns MOE_ERR_INVALID_ARG for a mode other than 0, a bad budget or a null timed_out; the
 * timeout itself is read with moe_get_error. */
MOE_API moe_status_t moe_selftest_wait_timeout(int32_t mode, int64_t budget_cycles, int32_t* timed_out,
                                               void* scratch, moe_stream_t stream);

/* Kernel trace: the device time of every kernel the library launches, for profiling from
 * the host without an external profiler. The pages have no counterpart.
 * moe_trace_begin opens a trace on the calling host thread, with room for max_launches
 * (1 .. 65536) launches; it creates 2 * max_launches CUDA timing events (no device memory)
 * and discards the previous trace's results. Until moe_trace_end, every kernel the library
 * launches from this thread, on a stream that is not being captured into a graph, is
 * bracketed by two events recorded on its own stream: the kernel then starts only after the
 * previous work of its stream has finished (no overlap with a dependent launch), so each
 * duration is the kernel's own; while a trace is open, moe_backward also keeps its two
 * branches from overlapping (its caller's stream waits for the side branch). Launches beyond
 * max_launches are not traced (counted by moe_trace_dropped).
 * moe_trace_end synchronises the recorded events and returns the number of traced launches
 * (>= 0), or MOE_ERR_INVALID_ARG if no trace is open, or MOE_ERR_CUDA.
 * moe_trace_record gives launch i's kernel name (without parameters, e.g.
 * "route_tc_kernel<2>"; the string stays valid until the next moe_trace_begin on this thread)
 * and its duration in milliseconds, in launch order. */
MOE_API moe_status_t moe_trace_begin(int32_t max_launches);
MOE_API int32_t moe_trace_end(void);
MOE_API moe_status_t moe_trace_record(int32_t i, const char** name, float* ms);
MOE_API int32_t moe_trace_dropped(void);

/* Static description of a status code (never NULL). */
MOE_API const char* moe_status_str(moe_status_t status);

/* Number of kernels this library has launched in this process (all devices). */
MOE_API uint64_t moe_kernel_launches(void);

/* Library version string, e.g. "moe-gb300 0.1 sm_103a". */
MOE_API const char* moe_version(void);

#ifdef __cplusplus
}
#endif
#endif /* MOE_H */
