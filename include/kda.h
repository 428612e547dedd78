/*
 * libkda -- Kimi Delta Attention (KDA) on one GB300 (sm_103a): packed prefill,
 * decode, ReplaySSM replay, state-pool operations, input preprocessing and the
 * short convolution, and the backward of the prefill; and, for the softmax
 * attention layers that a hybrid model has beside its KDA layers, one speculative
 * step: rotary positions, attention of a drafted tree over a paged cache,
 * verification of the drafted tokens, and the append of the accepted ones; and a
 * decoding step of samples that branch from shared prompts: per-head norms with
 * rotary positions, attention over the shared prefix joined with the samples' own
 * keys, and sampling from logits.
 *
 * What is computed.  The KDA paragraph of "Kimi K3 on Fireworks: Fast RL at
 * frontier scale" (kernels section) describes KDA as linear attention that
 * updates a compact, fixed-size recurrent state per head with channel-wise
 * gating, trained in chunk-parallel form.  The pages print no equation; this
 * library implements the gated delta rule with per-channel decay, for each
 * (sequence, head) with state S in R^{dk x dv}:
 *
 *     S <- Diag(exp(g_t)) S                    (decay of the dk rows)
 *     S <- S - beta_t k_t (k_t^T S) + beta_t k_t v_t^T
 *     o_t = S^T (scale * q_t)                  (output after the update)
 *
 * The same page's speculative-decoding paragraph (ReplaySSM) keeps the
 * recurrent state consistent after rejected draft tokens by replaying the
 * accepted tokens' update inputs from a committed checkpoint: kda_replay.
 *
 * Conventions shared by every call
 * --------------------------------
 * - All tensor arguments are DEVICE pointers to caller-owned memory (the
 *   state-pool offload / restore calls also take page-locked host memory).  The
 *   library never allocates or frees device memory; its scratch is the caller's
 *   workspace (kda_chunk_fwd_noalloc: one fixed array of its own).
 * - Token-major packed layouts, C-contiguous:
 *     q, k, g  [T, H, dk]     v, o [T, H, dv]     beta [T, H]
 *   of dtype `kda_dtype` (bf16 or fp32; o uses the same dtype as the inputs).
 *   States are always fp32, [.., H, dk, dv] with dv contiguous.
 * - g holds log-gates (alpha = exp(g) in [0, 1]); g = -inf erases the state.
 * - dk and dv must each be 64 or 128 (KDA_ERR_UNSUPPORTED otherwise).
 * - Pointers must be 16-byte aligned (beta: element-aligned; each call's
 *   section names its exceptions).
 * - `stream` is a cudaStream_t (NULL = legacy default stream).  Every call is
 *   asynchronous on `stream`; none synchronizes except kda_device_status.
 * - Errors the host can see (NULL pointers, bad sizes, dtype, alignment, small
 *   workspace) return immediately and launch nothing.  Errors only the device
 *   can see (bad cu_seqlens / cu_accept, slot out of range, gate range, a
 *   bounded wait that gave up) are OR-ed into a status word in the workspace;
 *   read it with kda_device_status.  Each call clears that word first.  A
 *   work item that detects a device error skips its work and writes nothing.
 *   No call aborts, prints or traps.
 * - Results are deterministic: fixed reduction order, no floating-point
 *   atomics; the same sequence gives the same bits whatever else is batched
 *   with it.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kda_status {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARGUMENT = 1, /* NULL pointer, negative size, misaligned pointer          */
    KDA_ERR_UNSUPPORTED = 2,      /* dk/dv not in {64,128}, unknown dtype                     */
    KDA_ERR_WORKSPACE = 3,        /* workspace NULL or smaller than required                  */
    KDA_ERR_CUDA = 4,             /* a CUDA runtime call or launch failed                     */
    KDA_ERR_GATE_RANGE = 5,       /* device: a chunk decays below 2^-100 and the workspace has
                                     no room to recompute its chain (see kda_chunk_fwd)       */
    KDA_ERR_TIMEOUT = 6,          /* device: a bounded wait gave up                           */
    KDA_ERR_BAD_SEQLENS = 7,      /* device: cu_seqlens / cu_accept not a valid partition     */
    KDA_ERR_BAD_SLOT = 8,         /* device: slot or row index outside its array              */
    KDA_ERR_BAD_PAGE = 9,         /* device: page index outside the pool, or a context longer
                                     than the block table                                     */
    KDA_ERR_BAD_TREE = 10         /* device: a drafted node's parent or token is not valid    */
} kda_status;

typedef enum kda_dtype {
    KDA_BF16 = 0, /* q, k, v, g, beta and o are bfloat16 */
    KDA_F32 = 1   /* q, k, v, g, beta and o are float32  */
} kda_dtype;

/* Bytes at the start of every workspace: the device status word and padding. */
#define KDA_WS_HEADER_BYTES 256

/*
 * Workspace for kda_chunk_fwd, in bytes: the size with which every path of the
 * call is available.  Returns 0 for invalid arguments.
 *
 * The minimum is smaller.  With final_state != NULL, KDA_WS_HEADER_BYTES
 * suffice; with final_state == NULL the chunked path needs a staging copy of
 * every (sequence, head) state (N*H*dk*dv*4 bytes after the header) to hand the
 * state from the chunked kernel to the partial-chunk kernel.
 *
 * T-segment split: when dk = dv = 128, N*H <= 48 and T_total >= 4096, a batch
 * has too few (sequence, head) chains to occupy the GPU, and kda_chunk_fwd cuts
 * the full chunks of every sequence in two at a chunk boundary and runs the
 * halves concurrently: segment 1 from a zero state and, with v = 0, from the
 * identity (its transition), then merges the results exactly (the recurrence is
 * affine in the state) -- the context-parallel hand-over of a long sequence's
 * state described in "Kimi K3 on Fireworks: Fast RL at frontier scale", done
 * within one GPU.  It needs 3*N*H*dk*dv*4 + T_total*H*dv*2 bytes after the
 * header, which this function then includes; with a smaller (but sufficient)
 * workspace the call runs unsplit.  Results agree within floating-point
 * rounding either way.
 *
 * Launch order: when a batch has more (sequence, head) chains than one wave of
 * chunked-kernel CTAs (N*H > 152, 2 <= N <= 8192, cu_seqlens given), the call
 * ranks the sequences by length on the device and starts the longest chains
 * first, which shortens the tail of a variable-length batch.  It needs N int32
 * (rounded up to 16 bytes) after the staging states, which this function then
 * includes; the results are bit-identical with or without it.  With it, chunked-kernel
 * CTAs are launched only for the first floor(T_total / 64) sequences of that order
 * (the others have no full chunk), which keeps a batch of short sequences (a
 * speculative verify step) from paying for thousands of empty CTAs.
 *
 * Strong decay: the chunked kernel factors each chunk's decay through prefix
 * products and needs every channel's product over a 64-token chunk to stay at or
 * above 2^-100.  With N*H bytes (rounded up to 16) after everything above, which
 * this function includes, a (sequence, head) chain that leaves that range is
 * flagged and recomputed from its initial state by the token-sequential kernel,
 * which takes any gate (g = -inf included); without that room the call reports
 * KDA_ERR_GATE_RANGE instead.
 */
size_t kda_chunk_fwd_workspace_size(int N, int64_t T_total, int H, int dk, int dv);

/*
 * Packed variable-length prefill (the chunk-parallel training/prefill form).
 *
 *   q, k, g      [T_total, H, dk]   dtype
 *   v            [T_total, H, dv]   dtype
 *   beta         [T_total, H]       dtype
 *   init_state   [N, H, dk, dv] fp32, or NULL for zeros
 *   cu_seqlens   [N+1] int32 on the device, cu[0] = 0, non-decreasing,
 *                cu[N] = T_total; sequence n is tokens [cu[n], cu[n+1]).
 *                NULL means N sequences of equal length T_total / N.
 *   scale        multiplies q (pass 1/sqrt(dk) for raw queries)
 *   o            [T_total, H, dv]   dtype (written for every token)
 *   final_state  [N, H, dk, dv] fp32, or NULL (not written).  May alias
 *                init_state (in-place update).
 *   workspace    >= kda_chunk_fwd_workspace_size() bytes (see above), device.
 *
 * Full 64-token chunks run through the chunked WY kernel (bf16; dk and dv each
 * 64 or 128: the kernel's tiles are 128 wide and a 64-wide head arrives with
 * zero channels and columns, which leave the result unchanged);
 * the last len % 64 tokens of each sequence, sequences shorter than 64, and
 * fp32 inputs run through the token-sequential kernel,
 * which is the same routine kda_decode_step and kda_replay use: a 1-token
 * sequence here gives the same bits as kda_decode_step on the same state.
 * An empty sequence copies init_state to final_state.  A chain whose chunk
 * decays below the chunked kernel's range is recomputed token by token (see
 * kda_chunk_fwd_workspace_size), so any gate values are accepted.
 */
kda_status kda_chunk_fwd(const void *q, const void *k, const void *v, const void *g, const void *beta,
                         kda_dtype dtype, const float *init_state, const int32_t *cu_seqlens, int N,
                         int64_t T_total, int H, int dk, int dv, float scale, void *o, float *final_state,
                         void *workspace, size_t ws_bytes, void *stream);

/*
 * Optional input preprocessing, fused into the kernels (the kda_*_prep calls):
 * callers that hold raw projections pass them as they are and skip a separate
 * normalisation pass over q, k, g and beta.  The pages do not define KDA's
 * input maps; the common ones for delta-rule attention are provided, each
 * behind its own flag:
 *   KDA_PREP_L2NORM_Q     q_t <- q_t / sqrt(sum_i q_{t,i}^2 + l2_eps)   per (token, head)
 *   KDA_PREP_L2NORM_K     k_t <- k_t / sqrt(sum_i k_{t,i}^2 + l2_eps)
 *   KDA_PREP_SIGMOID_GATE g holds raw gates x: the log-gate is logsigmoid(x), so the
 *                         decay is alpha = sigmoid(x) (0 only where fp32 underflows,
 *                         below about x = -88)
 *   KDA_PREP_SIGMOID_BETA beta <- sigmoid(beta)
 * scale still multiplies q after the normalisation.  Unknown flags or a
 * negative / non-finite l2_eps return KDA_ERR_INVALID_ARGUMENT.  With prep = 0
 * the _prep calls are exactly the plain ones.
 */
#define KDA_PREP_L2NORM_Q 1u
#define KDA_PREP_L2NORM_K 2u
#define KDA_PREP_SIGMOID_GATE 4u
#define KDA_PREP_SIGMOID_BETA 8u

kda_status kda_chunk_fwd_prep(const void *q, const void *k, const void *v, const void *g, const void *beta,
                              kda_dtype dtype, const float *init_state, const int32_t *cu_seqlens, int N,
                              int64_t T_total, int H, int dk, int dv, float scale, uint32_t prep, float l2_eps,
                              void *o, float *final_state, void *workspace, size_t ws_bytes, void *stream);

/*
 * One decode token per sequence on a slot-indexed state pool (in place).
 *
 *   q, k, g      [N, H, dk]   dtype;  v [N, H, dv];  beta [N, H]
 *   state_pool   [num_slots, H, dk, dv] fp32, read and written in place
 *   slots        [N] int32 device, or NULL for slot n = n (needs N <= num_slots).
 *                Two sequences must not name the same slot.
 *   o            [N, H, dv]   dtype
 *   workspace    >= KDA_WS_HEADER_BYTES bytes (status word)
 */
kda_status kda_decode_step(const void *q, const void *k, const void *v, const void *g, const void *beta,
                           kda_dtype dtype, float *state_pool, int64_t num_slots, const int32_t *slots,
                           int N, int H, int dk, int dv, float scale, void *o, void *workspace,
                           size_t ws_bytes, void *stream);

/* kda_decode_step with input preprocessing (see kda_chunk_fwd_prep). */
kda_status kda_decode_step_prep(const void *q, const void *k, const void *v, const void *g, const void *beta,
                                kda_dtype dtype, float *state_pool, int64_t num_slots, const int32_t *slots,
                                int N, int H, int dk, int dv, float scale, uint32_t prep, float l2_eps, void *o,
                                void *workspace, size_t ws_bytes, void *stream);

/*
 * ReplaySSM-style rollback: apply each sequence's accepted tokens to its
 * committed state, in place, without producing outputs.  Equivalent to
 * kda_chunk_fwd over the accepted tokens with init_state = final_state =
 * the committed state (bit for bit).
 *
 *   state_pool   [num_slots, H, dk, dv] fp32, in place
 *   slots        [N] int32 device, or NULL for slot n = n
 *   k, g         [A_total, H, dk] dtype;  v [A_total, H, dv];  beta [A_total, H]
 *   cu_accept    [N+1] int32 device; sequence n's accepted tokens are
 *                [cu_accept[n], cu_accept[n+1]) (0 tokens leaves the state)
 *   workspace    >= KDA_WS_HEADER_BYTES bytes (status word)
 */
kda_status kda_replay(float *state_pool, int64_t num_slots, const int32_t *slots, const void *k,
                      const void *v, const void *g, const void *beta, kda_dtype dtype,
                      const int32_t *cu_accept, int N, int64_t A_total, int H, int dk, int dv,
                      void *workspace, size_t ws_bytes, void *stream);

/*
 * State-pool operations for rollout caching.  In RL rollouts many trajectories
 * branch from a shared prompt, and each branch continues from its own copy of
 * the prompt's recurrent state; the states of inactive trajectories are kept
 * in host memory and brought back when the trajectory resumes ("Kimi K3 on
 * Fireworks: Fast RL at frontier scale": the rollout paragraph on MLA / KDA
 * histories that stay consistent as trajectories branch from shared prompts,
 * and the serverless-training paragraph on moving reusable KV and KDA states to
 * host memory and loading inactive snapshots asynchronously).
 *
 * A slot's state is the whole [H, dk, dv] fp32 block of the pool,
 * state_pool[slot] (H*dk*dv*4 bytes).  Slot arrays are int32 DEVICE arrays of
 * length n.  A slot outside [0, num_slots) sets KDA_ERR_BAD_SLOT in the status
 * word and that item copies nothing.  Copies are exact (bit for bit).
 * workspace: >= KDA_WS_HEADER_BYTES bytes (status word).
 */

/* Fork: state_pool[dst_slots[i]] = state_pool[src_slots[i]] for i < n.  No
 * destination may appear twice or be the source of another item (the items
 * run concurrently); src == dst copies a state onto itself. */
kda_status kda_state_fork(float *state_pool, int64_t num_slots, const int32_t *src_slots, const int32_t *dst_slots,
                          int n, int H, int dk, int dv, void *workspace, size_t ws_bytes, void *stream);

/* Offload: host_states[i] = state_pool[slots[i]] (slots NULL: slot i), for i < n.
 * host_states: [n, H, dk, dv] fp32 in page-locked host memory that the device
 * can address (cudaHostAlloc / cudaHostRegister with mapping; with unified
 * addressing every page-locked allocation is), 16-byte aligned; otherwise
 * KDA_ERR_INVALID_ARGUMENT.  The kernel writes the host memory directly;
 * synchronize `stream` before reading it on the host. */
kda_status kda_state_offload(const float *state_pool, int64_t num_slots, const int32_t *slots, int n, int H, int dk,
                             int dv, float *host_states, void *workspace, size_t ws_bytes, void *stream);

/* Restore: state_pool[slots[i]] = host_states[i] (slots NULL: slot i), for i < n;
 * host_states as for kda_state_offload.  No slot may appear twice. */
kda_status kda_state_restore(float *state_pool, int64_t num_slots, const int32_t *slots, int n, int H, int dk,
                             int dv, const float *host_states, void *workspace, size_t ws_bytes, void *stream);

/* kda_replay with input preprocessing (see kda_chunk_fwd_prep; KDA_PREP_L2NORM_Q has
 * no effect, replay reads no q).  Bit for bit the final state of
 * kda_chunk_fwd_prep over the accepted tokens with the same flags. */
kda_status kda_replay_prep(float *state_pool, int64_t num_slots, const int32_t *slots, const void *k,
                           const void *v, const void *g, const void *beta, kda_dtype dtype,
                           const int32_t *cu_accept, int N, int64_t A_total, int H, int dk, int dv, uint32_t prep,
                           float l2_eps, void *workspace, size_t ws_bytes, void *stream);

/*
 * Backward of kda_chunk_fwd (training): the gradients of a loss with respect to
 * q, k, v, g (the log-gates), beta and the initial states, given its gradients
 * with respect to o (d_o [T_total, H, dv]) and to the final states
 * (d_final_state [N, H, dk, dv] fp32, or NULL = zero).  The KDA paragraph of
 * "Kimi K3 on Fireworks: Fast RL at frontier scale" quotes a backward kernel but
 * no formula; this is the reverse mode of the same recurrence, evaluated on the
 * 64-token chunked form in four launches: a forward pass stores the state at
 * every chunk start in the workspace; every (chunk, head) computes its
 * chunk-local terms in parallel; one CTA per (sequence, head, block of state
 * columns) carries the state gradient back through the chunks; every (chunk,
 * head) then computes its gradients in parallel.  The matrix products run on the
 * tensor cores in tf32 with fp32 accumulation.  Gates whose 64-token decay falls
 * below the chunked form's range are not recomputed token by token here (the
 * forward call does that): the backward reports KDA_ERR_GATE_RANGE instead.
 *
 * Inputs as for kda_chunk_fwd (same dtype, layouts, cu_seqlens, init_state,
 * scale).  Outputs, all in the input dtype: d_q, d_k, d_g [T_total, H, dk],
 * d_v [T_total, H, dv], d_beta [T_total, H]; d_init_state [N, H, dk, dv] fp32 or
 * NULL.  Every output element is written (they need no clearing).
 * Workspace: at least kda_chunk_bwd_workspace_size(N, T_total, H, dk, dv) bytes,
 * 16-byte aligned, owned by the caller, not read back.  Errors as for
 * kda_chunk_fwd: KDA_ERR_UNSUPPORTED (dtype, dk, dv), KDA_ERR_INVALID_ARGUMENT
 * (NULL or misaligned pointers, N not dividing T_total without cu_seqlens),
 * KDA_ERR_WORKSPACE; invalid cu_seqlens and a chunk decay below 2^-100 are
 * reported through kda_device_status (KDA_ERR_BAD_SEQLENS, KDA_ERR_GATE_RANGE).
 */
size_t kda_chunk_bwd_workspace_size(int N, int64_t T_total, int H, int dk, int dv);

kda_status kda_chunk_bwd(const void *q, const void *k, const void *v, const void *g, const void *beta,
                         kda_dtype dtype, const float *init_state, const int32_t *cu_seqlens, int N,
                         int64_t T_total, int H, int dk, int dv, float scale, const void *d_o,
                         const float *d_final_state, void *d_q, void *d_k, void *d_v, void *d_g, void *d_beta,
                         float *d_init_state, void *workspace, size_t ws_bytes, void *stream);

/* kda_chunk_bwd for a forward taken with kda_chunk_fwd_prep: the inputs are the raw
 * ones given to the forward, with the same prep flags and l2_eps, and the gradients
 * are taken with respect to those raw inputs (carried back through the L2
 * normalisation, alpha = sigmoid(x_g) and beta = sigmoid(x_beta)).  prep = 0 is
 * kda_chunk_bwd. */
kda_status kda_chunk_bwd_prep(const void *q, const void *k, const void *v, const void *g, const void *beta,
                              kda_dtype dtype, const float *init_state, const int32_t *cu_seqlens, int N,
                              int64_t T_total, int H, int dk, int dv, float scale, uint32_t prep, float l2_eps,
                              const void *d_o, const float *d_final_state, void *d_q, void *d_k, void *d_v,
                              void *d_g, void *d_beta, float *d_init_state, void *workspace, size_t ws_bytes,
                              void *stream);

/*
 * Short convolution of the input projections, with its state carried across calls
 * (the disaggregated-serving paragraph of "Kimi K3 on Fireworks: Fast RL at
 * frontier scale" lists KDA's convolution state beside its recurrent state; the
 * pages define neither).  The reading implemented: a depthwise causal convolution
 * of width KDA_CONV_WIDTH over the tokens of each sequence, one weight vector per
 * channel, then SiLU:
 *   pre_t[c] = sum_{i=0}^{3} w[h][c][i] x_{t-3+i}[c],   y_t[c] = pre / (1 + exp(-pre)),
 * applied to q, k and v before everything else (the _prep flags act on its output).
 * Channels of a head are packed (q 0..dk-1 | k dk..2dk-1 | v 2dk..2dk+dv-1):
 *   conv_weight [H, 2dk+dv, KDA_CONV_WIDTH] fp32;
 *   a convolution state [KDA_CONV_WIDTH-1, H, 2dk+dv] fp32 per sequence holds its
 *   previous raw inputs, oldest first (zeros for a new sequence).
 *
 * kda_conv_fwd: the prefill form.  q, k, v [T_total, H, d] raw -> q_out, k_out,
 * v_out (same dtype and layout, not overlapping the inputs, since a block's window
 * reads the raw rows before it; then call kda_chunk_fwd(_prep) on them);
 * conv_state_in / conv_state_out [N, 3, H, 2dk+dv] (either NULL = zeros / not
 * written; they may be the same buffer).
 * kda_decode_step_conv / kda_replay_conv: the decode and replay forms, the
 * convolution fused into the token-sequential kernel; conv_pool [num_slots, 3, H,
 * 2dk+dv] is indexed by the same slots as state_pool and advanced in place.  Replay
 * takes q too: the accepted tokens' q advances the convolution state.
 * conv_width must be KDA_CONV_WIDTH (else KDA_ERR_UNSUPPORTED); other errors as
 * for the calls without convolution.
 */
#define KDA_CONV_WIDTH 4

kda_status kda_conv_fwd(const void *q, const void *k, const void *v, kda_dtype dtype, const float *conv_weight,
                        int conv_width, const float *conv_state_in, const int32_t *cu_seqlens, int N, int64_t T_total,
                        int H, int dk, int dv, void *q_out, void *k_out, void *v_out, float *conv_state_out,
                        void *workspace, size_t ws_bytes, void *stream);

kda_status kda_decode_step_conv(const void *q, const void *k, const void *v, const void *g, const void *beta,
                                kda_dtype dtype, float *state_pool, int64_t num_slots, const int32_t *slots,
                                int N, int H, int dk, int dv, float scale, const float *conv_weight,
                                int conv_width, float *conv_pool, uint32_t prep, float l2_eps, void *o,
                                void *workspace, size_t ws_bytes, void *stream);

kda_status kda_replay_conv(float *state_pool, int64_t num_slots, const int32_t *slots, const void *q, const void *k,
                           const void *v, const void *g, const void *beta, kda_dtype dtype,
                           const int32_t *cu_accept, int N, int64_t A_total, int H, int dk, int dv,
                           const float *conv_weight, int conv_width, float *conv_pool, uint32_t prep, float l2_eps,
                           void *workspace, size_t ws_bytes, void *stream);

/*
 * One speculative step of a softmax-attention layer.  A hybrid model interleaves
 * KDA layers with attention layers whose keys and values are cached, and both have
 * to represent the same prefix ("Kimi K3 on Fireworks: Fast RL at frontier scale":
 * the KV-cache and speculative-decoding paragraphs).  The calls below give the
 * attention layers what kda_chunk_fwd + kda_replay give the KDA layers: the drafted
 * tokens attend to the cache without entering it (kda_tree_attn), verification
 * decides which of them stand (kda_draft_verify), and only those are applied, by
 * kda_replay to the recurrent states and by kda_cache_append to the cache.
 *
 * Drafted trees.  Sequence n of N has the nodes [cu_nodes[n], cu_nodes[n+1]) of the
 * packed node arrays, at most KDA_MAX_TREE_NODES.  Node 0 is the root: the token
 * that follows the committed context (already sampled).  parent[i] is the local
 * index of a node's parent, 0 <= parent[i] < i (the root's entry is not read);
 * parent NULL means chains, parent[i] = i - 1.  cu_nodes [N+1] int32 on the device:
 * cu_nodes[0] = 0, non-decreasing, cu_nodes[N] <= the number of packed nodes.  Where it
 * is not, a sequence whose own two entries are out of range or decrease, or that
 * begins before an earlier entry, is reported as KDA_ERR_BAD_SEQLENS and left out;
 * the others are worked on.
 */
#define KDA_MAX_TREE_NODES 64

/*
 * Rotary positions of q and k.  Pair j < rot/2 of a head's channels -- (j, j + rot/2),
 * or (2j, 2j + 1) with interleaved != 0 -- at position p turns by the angle
 * t = p * inv_freq[j]:
 *     (a, b) -> mscale (a cos t - b sin t, a sin t + b cos t);
 * the channels from rot on are copied.  kda_rope_bwd is its gradient (the transposed
 * map: the angle's sign changes), with the output gradients in place of q and k.
 *   q, k        [T, Hq, d], [T, Hk, d] dtype; token t of q starts q_stride elements
 *               after token t - 1 (0: Hq * d); k likewise.  k NULL or Hk = 0: q only.
 *   positions   [T] int32 (any value)      inv_freq [rot/2] fp64, radians per position
 *   q_out,k_out as q, k with their own strides; may be q and k themselves (same stride).
 * d: a multiple of 8, at most 1024; rot even, 0 <= rot <= d.  Angles are reduced in
 * 64-bit fixed point and are off by at most |p inv_freq| 2^-52 radians (about what
 * rounding inv_freq to fp64 costs); sines, cosines and products are fp32, the result is
 * rounded to dtype once.
 * Pointers are element-aligned; 16-byte aligned rows (and rot / 2, or interleaved rot,
 * a multiple of 16 bytes) take the vector path.  Nothing to report from the device,
 * so no workspace.
 */
kda_status kda_rope(const void *q, const void *k, kda_dtype dtype, const int32_t *positions, const double *inv_freq,
                    int64_t T, int Hq, int Hk, int d, int rot, int64_t q_stride, int64_t k_stride, int interleaved,
                    float mscale, void *q_out, void *k_out, int64_t q_out_stride, int64_t k_out_stride, void *stream);
kda_status kda_rope_bwd(const void *d_q_out, const void *d_k_out, kda_dtype dtype, const int32_t *positions,
                        const double *inv_freq, int64_t T, int Hq, int Hk, int d, int rot, int64_t q_stride,
                        int64_t k_stride, int interleaved, float mscale, void *d_q, void *d_k, int64_t q_out_stride,
                        int64_t k_out_stride, void *stream);

/*
 * A paged cache of keys and values: key row r of page p for head h starts at
 * k + p * k_page_stride + r * k_row_stride + h * k_head_stride (elements; any order
 * of the axes), its dk channels contiguous; values likewise.  Strides and pointers
 * are multiples of 16 bytes.  Row r of sequence n lies in page
 * block_table[n * table_stride + r / page_size], slot r % page_size; its committed
 * context is rows [0, ctx_len[n]).  All pointers are device pointers, the struct
 * itself is read on the host during the call.
 */
typedef struct kda_paged_kv {
    void *k, *v;
    int64_t k_page_stride, k_row_stride, k_head_stride;
    int64_t v_page_stride, v_row_stride, v_head_stride;
    int64_t num_pages;
    int64_t table_stride;
    const int32_t *block_table; /* [N, max_pages] int32 */
    const int32_t *ctx_len;     /* [N] int32 */
    int page_size, max_pages;
} kda_paged_kv;

/*
 * Attention of drafted trees over a paged cache: node i of sequence n attends to the
 * sequence's context rows, to its ancestors and to itself (a one-node tree is the plain
 * decode step).  Query head h reads KV head h / (Hq / Hkv).
 *   q      [T, Hq, dk] dtype, token stride q_stride elements (0: packed)
 *   k, v   [T, Hkv, dk], [T, Hkv, dv]: the nodes' own keys and values, not in the cache
 *   o      [T, Hq, dv] dtype, packed;  lse [T, Hq] fp32 or NULL: log sum exp(scale q.k)
 *   max_nodes  the largest tree of the batch (1..KDA_MAX_TREE_NODES); a larger one is
 *          reported as KDA_ERR_BAD_SEQLENS.  A bound far above the trees costs workspace
 *          and, where it allows more than 32 rows per KV head in bf16, two launches.  T <= N * max_nodes; packed nodes from
 *          cu_nodes[N] on are not read, and their outputs not written.
 * dk, dv each 64 or 128; page_size * max_pages < 2^31.  Scores, softmax and sums are fp32; for bf16 the weights are
 * rounded to bf16 (by at most 2^-8 of each) before they meet the values, as the tensor cores take both operands in one
 * type (fp32 inputs: products in three tf32 terms, about 22 bits).
 * A node's infinities and NaN reach the rows that see the node, and no others.
 * Long contexts are cut into parts that run concurrently and are joined in a fixed
 * order; the cut goes by a sequence's own length and tree, so its bits do not depend
 * on the batch.  A sequence with a device error (BAD_SEQLENS, BAD_PAGE, BAD_TREE)
 * writes nothing.
 */
size_t kda_tree_attn_workspace_size(int N, int64_t T, int Hq, int Hkv, int dv, int max_nodes, int64_t max_ctx);
/* The same for one type (bf16's is the smaller where trees are small). */
size_t kda_tree_attn_workspace_size_for(kda_dtype dtype, int N, int64_t T, int Hq, int Hkv, int dv, int max_nodes,
                                        int64_t max_ctx);

kda_status kda_tree_attn(const void *q, const void *k, const void *v, kda_dtype dtype, const kda_paged_kv *cache,
                         const int32_t *cu_nodes, const int32_t *parent, int N, int64_t T, int Hq, int Hkv, int dk,
                         int dv, int64_t q_stride, int64_t k_stride, int64_t v_stride, int max_nodes, float scale,
                         void *o, float *lse, void *workspace, size_t ws_bytes, void *stream);

/*
 * Append rows to a paged cache: rows j in [cu[n], cu[n+1]) go to positions
 * ctx_len[n] + j - cu[n] of sequence n.  Row j is row `rows[j]` of k and v, or row j
 * with rows NULL: kda_draft_verify's cu_accept and rows append the accepted nodes of a
 * drafted tree.  cu [N+1] as cu_nodes above; A_total >= cu[N] is the number of rows
 * given (the rest are not read).  k, v: T_src rows, strides as for kda_tree_attn.
 *   new_len  [N] int32 or NULL: ctx_len[n] + cu[n+1] - cu[n]; must not be ctx_len itself
 * Device errors: BAD_SEQLENS, and BAD_PAGE for a sequence that does not fit its block
 * table: such a sequence keeps its length and writes nothing.  BAD_PAGE for a row whose
 * page is outside the pool and BAD_SLOT for rows[j] outside [0, T_src): that row is not
 * written, but the others are and new_len counts it, so after these two errors the
 * length covers a row that was never stored.  Two rows must not name the same place.
 * workspace: >= KDA_WS_HEADER_BYTES.
 */
kda_status kda_cache_append(const void *k, const void *v, kda_dtype dtype, const kda_paged_kv *cache,
                            const int32_t *cu, const int32_t *rows, int N, int64_t A_total, int64_t T_src, int Hkv,
                            int dk, int dv, int64_t k_stride, int64_t v_stride, int32_t *new_len, void *workspace,
                            size_t ws_bytes, void *stream);

/*
 * Verification of drafted trees against the target model's probabilities, from given
 * uniform numbers in [0, 1).  The walk starts at the root.  At a node with target row p
 * and draft row q its children are tried in index order; with A = 0, R = 1 and the
 * residual r_v = max(0, p_v - A q_v), a child with token x and number u is accepted if
 *     u q_x R < r_x,
 * else A += R and R = sum_v r_v.  (That is repeated rejection sampling: the residual
 * after a refusal is max(0, r - R q) up to its mass, and max(0, max(0, a) - b) =
 * max(0, a - b) leaves one scalar for all refusals.)  Without draft probabilities the
 * drafts are taken as certain: accepted if u R < r_x, else R -= r_x and r_x = 0.  When
 * no child is accepted the next token is drawn from r by u_sample: the lowest v with
 * sum_{w <= v} r_w > u_sample sum_w r_w.  A residual without mass leaves p in its place;
 * p without mass gives token -1.  NaN counts as no mass.
 *   tokens       [T] int32: the nodes' tokens (the root's is not read)
 *   target_probs [T, V] dtype, row stride target_stride elements (0: V): row i is the
 *                target's distribution after node i
 *   draft_probs  [T, V] dtype (draft_stride) or NULL: row i is the distribution that
 *                node i's children were drawn from
 *   u_accept     [T] fp32 (the root's is not read)      u_sample [N] fp32
 * Outputs: cu_accept [N+1] int32: sequence n accepts cu_accept[n+1] - cu_accept[n] nodes,
 * the root among them; rows [T] int32: their packed indices in order, -1 from
 * cu_accept[N] on; next_token [N] int32.  (cu_accept and the rows' k, v, g, beta are what
 * kda_replay takes; it wants exactly cu_accept[N] tokens, so the caller reads that count on
 * the host before it gathers them.  kda_cache_append takes cu_accept and rows as they are.)
 * An empty tree, or one with a device error (BAD_SEQLENS, BAD_TREE),
 * accepts nothing and gives token -1.
 * p - A q and its sums are carried to about 1e-13 (pairs of fp32; fp64 for the walk's
 * scalars), so a decision stands unless a number lies that close to a border.
 * V: at most 2^24.  workspace: >= kda_draft_verify_workspace_size(N).
 */
size_t kda_draft_verify_workspace_size(int N);

kda_status kda_draft_verify(const int32_t *tokens, const int32_t *cu_nodes, const int32_t *parent,
                            const void *target_probs, const void *draft_probs, kda_dtype dtype, const float *u_accept,
                            const float *u_sample, int N, int64_t T, int V, int64_t target_stride,
                            int64_t draft_stride, int32_t *cu_accept, int32_t *rows, int32_t *next_token,
                            void *workspace, size_t ws_bytes, void *stream);

/* ---- a decoding step of branching rollouts, beside the speculative step above ---- */

/*
 * RMS norm of every head of q and k with learned weights, then rotary positions, in one
 * pass: with n = x / sqrt(mean_i x_i^2 + eps) over a head's d channels, a head becomes
 * kda_rope of weight * n (mscale multiplies the rotated channels only).  Arguments as for
 * kda_rope, and
 *   q_weight, k_weight  [d] of weight_dtype, or NULL: ones
 *   eps   finite, >= 0
 * Norms, weights, sines and products are fp32 (the squares of a head and their mean have to lie
 * within its range); the result is rounded to dtype once.  q_out and k_out may be q and k
 * themselves (same stride).
 *
 * kda_norm_rope_bwd is the gradient: from q, k (the inputs of the forward) and the gradients
 * of its outputs to d_q, d_k and, where not NULL, d_q_weight, d_k_weight [d] fp32 (sums over
 * all tokens and heads, in a fixed order; always fp32, as a sum of T * H terms needs them, and
 * with an error that does not grow with T * H).
 * d_q may be d_q_out or q itself (same stride), d_k likewise.
 * workspace: >= kda_norm_rope_bwd_workspace_size(d) bytes, 16-byte aligned; nothing to report
 * from the device.
 */
kda_status kda_norm_rope(const void *q, const void *k, kda_dtype dtype, const void *q_weight, const void *k_weight,
                         kda_dtype weight_dtype, const int32_t *positions, const double *inv_freq, int64_t T, int Hq,
                         int Hk, int d, int rot, int64_t q_stride, int64_t k_stride, int interleaved, float mscale,
                         float eps, void *q_out, void *k_out, int64_t q_out_stride, int64_t k_out_stride, void *stream);

size_t kda_norm_rope_bwd_workspace_size(int d);

kda_status kda_norm_rope_bwd(const void *q, const void *k, const void *d_q_out, const void *d_k_out, kda_dtype dtype,
                             const void *q_weight, const void *k_weight, kda_dtype weight_dtype,
                             const int32_t *positions, const double *inv_freq, int64_t T, int Hq, int Hk, int d, int rot,
                             int64_t q_stride, int64_t k_stride, int64_t d_q_out_stride, int64_t d_k_out_stride,
                             int interleaved, float mscale, float eps, void *d_q, void *d_k, int64_t d_q_stride,
                             int64_t d_k_stride, float *d_q_weight, float *d_k_weight, void *workspace, size_t ws_bytes,
                             void *stream);

/*
 * Attention of groups of sequences over the prefix that each group shares (several samples of one
 * prompt): every token of group g attends to all rows of the group's prefix, whose keys and
 * values are read once for all of them, and the result is joined with what the tokens
 * have from their own keys (kda_tree_attn over each sequence's own pages gives o_tail and lse_tail).
 *   q         [T, Hq, dk] dtype, token stride q_stride elements (0: packed); query head h reads KV head h / (Hq / Hkv)
 *   prefixes  the paged cache with one block table row and one length (ctx_len) per group; keys of one page must
 *             not overlap (a row stride of at least dk or dv where a page has more than one row)
 *   cu_tokens [N+1] int32: group g has the packed tokens [cu_tokens[g], cu_tokens[g+1])
 *   o_tail    [T, Hq, dv] dtype, lse_tail [T, Hq] fp32, packed: the attention result and log-sum over other keys, or both
 *             NULL; a token whose lse_tail is -inf has no such keys and its o_tail is not read
 *   o         [T, Hq, dv] dtype, packed (may be o_tail);  lse [T, Hq] fp32 or NULL (may be lse_tail): log sum exp over both
 * A row without any key has o = 0 and lse = -inf.  Calls can be chained (a prefix of prefixes): a result is the next one's tail.
 * dk, dv each 64 or 128; page_size * max_pages < 2^31.  Packed tokens from cu_tokens[N] on do not matter, and their outputs are not
 * written.  Scores, softmax and sums are fp32 up to the one rounding of o; for bf16 the weights are rounded to bf16 (by at
 * most 2^-8 of each) before they meet the values.  The work is cut by the sizes of the whole batch, so the bits of a result depend on
 * them, but not on chance.
 * Device errors: BAD_SEQLENS, BAD_PAGE (a page outside the pool, or a prefix longer than its table row); such a group
 * writes nothing.  workspace: >= kda_prefix_attn_workspace_size(N, T, Hq, Hkv, dv) bytes, 16-byte aligned.
 */
size_t kda_prefix_attn_workspace_size(int N, int64_t T, int Hq, int Hkv, int dv);

kda_status kda_prefix_attn(const void *q, kda_dtype dtype, const kda_paged_kv *prefixes, const int32_t *cu_tokens, int N,
                           int64_t T, int Hq, int Hkv, int dk, int dv, int64_t q_stride, float scale, const void *o_tail,
                           const float *lse_tail, void *o, float *lse, void *workspace, size_t ws_bytes, void *stream);

/*
 * Sampling from logits by given uniform numbers, and the filtered distributions.  With M the
 * row's largest logit, e_i = exp((l_i - M) / temperature), and the tokens ordered by logit
 * (larger first), then by index (lower first):
 *   top_k   keeps the first top_k tokens (<= 0 or >= V: all);
 *   top_p   of these, the shortest run whose mass reaches top_p of theirs, at least one token
 *           (1 or more, or NaN: all);
 *   min_p   of these, the e_i >= min_p (<= 0 or NaN: all; 1 or more: the largest only).
 * token[n] is the lowest kept index i with sum_{kept j <= i} e_j > u[n] sum_{kept} e_j, and
 * probs[n] the kept e_i over their sum, zero elsewhere (and where fp32 has nothing so small): what
 * kda_draft_verify takes as target_probs or draft_probs.  A temperature that is not above 1e-30 (0,
 * negative, NaN) takes the lowest index of the largest logit; one above 1e30 counts as 1e30.  -inf
 * and NaN are never drawn; +inf counts as one value above all others.  A row without any other
 * logit gives token -1 and a distribution of zeros.  u is taken into [0, 1).
 *   logits  [N, V] dtype, row stride logits_stride elements (0: V)
 *   u       [N] fp32 (may be NULL without token)
 *   temperature, top_p, min_p [N] fp32, top_k [N] int32, each or NULL: 1, and no filter
 *   token   [N] int32 or NULL;  probs [N, V] of probs_dtype, row stride probs_stride (0: V), or NULL; one of
 *           them is given
 * The borders and the draw go by masses: whole numbers of 2^-44 of the largest for up to 2^19 tokens,
 * of twice as much whenever V is twice as large.  Each is good to 2e-10 of itself and half a unit, and
 * they are summed exactly.  So a decision stands unless a number lies within 2e-10 and V half units of
 * a border (2^-26 of the largest at 2^19 tokens, 2^-16 at 2^24), and a token of less than half a unit
 * is never drawn, though probs has its e.  The result does not depend on the batch.  V: at most 2^24.
 * Nothing to report from the device, so no workspace.
 */
kda_status kda_sample(const void *logits, kda_dtype dtype, const float *u, const float *temperature,
                      const int32_t *top_k, const float *top_p, const float *min_p, int N, int V, int64_t logits_stride,
                      int32_t *token, void *probs, kda_dtype probs_dtype, int64_t probs_stride, void *stream);

/*
 * Synchronizes `stream`, then reads the device status word of `workspace`
 * (errors from the last call that used it).  Returns KDA_OK or the first of
 * BAD_SEQLENS, BAD_SLOT, GATE_RANGE, TIMEOUT, BAD_PAGE, BAD_TREE that was raised; KDA_ERR_CUDA if
 * the synchronization or the copy failed.
 */
kda_status kda_device_status(const void *workspace, void *stream);

/* Size of the library-owned scratch behind kda_chunk_fwd_noalloc: the status
 * header plus staging room for 128 states of 128 x 128 fp32 (8 MiB). */
#define KDA_NOALLOC_WORKSPACE_BYTES ((size_t)KDA_WS_HEADER_BYTES + (size_t)8 * 1024 * 1024)

/*
 * kda_chunk_fwd for callers that cannot allocate device memory.  The pages
 * have no counterpart to this call: it exists for hosts that plan every device
 * byte themselves and give plug-in kernels no workspace hook, and for
 * latency-critical loops where a cudaMalloc (which can synchronize the device)
 * is not allowed.  It computes exactly what kda_chunk_fwd computes, with the
 * same arguments minus the workspace, and calls no allocator.
 *
 * Scratch: one array of KDA_NOALLOC_WORKSPACE_BYTES in the library's own
 * device memory; every GPU that loads libkda holds it until the process exits.
 * - Each call made outside stream capture looks up the array's device
 *   address on the current device; a call made during capture reuses the
 *   address last looked up there, so make the first call on a device before
 *   any stream capture (it returns KDA_ERR_CUDA otherwise).
 * - Every call shares the array: calls that could run at the same time on the
 *   GPU (other streams, other host threads on the same device) race on it and
 *   must be serialized by the caller.  The status word is cleared by each call.
 * - With final_state != NULL the size limit below does not apply and any
 *   batch is accepted.  With final_state == NULL the states are staged in the
 *   array, so N*H*dk*dv*4 must not exceed 8 MiB; larger requests return
 *   KDA_ERR_WORKSPACE and launch nothing.
 * - The call hands the whole array to kda_chunk_fwd as its workspace, so
 *   whatever of that call's optional buffers fit (the T-segment split's
 *   buffers, the launch order) are placed in the array too; overlapping calls
 *   race on all of it, not only on the status word and staged states.
 *
 *   status_workspace  optional out: receives the array's device address, which
 *                     kda_device_status() accepts to read this call's status.
 */
kda_status kda_chunk_fwd_noalloc(const void *q, const void *k, const void *v, const void *g, const void *beta,
                                 kda_dtype dtype, const float *init_state, const int32_t *cu_seqlens, int N,
                                 int64_t T_total, int H, int dk, int dv, float scale, void *o, float *final_state,
                                 const void **status_workspace, void *stream);

/*
 * 1 if kda_chunk_fwd runs its full 64-token chunks on the tensor-core (tcgen05)
 * kernel for this shape and dtype, 0 if every token goes through the
 * token-sequential kernel.  Pure query; touches no device.
 */
int kda_chunk_fwd_uses_tensor_cores(int dk, int dv, kda_dtype dtype);

/* Static, human-readable name of a status code. */
const char *kda_status_string(kda_status status);

/* Library version: major*10000 + minor*100 + patch. */
int kda_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
