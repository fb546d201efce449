/*
 * linattn.h -- C ABI of the GB300 (sm_103a) kernelized linear-attention library.
 *
 * The method ("Transformers are RNNs", as explained on wkq9411.github.io,
 * "【论文解读】Transformers are RNNs"): with phi(x) = elu(x) + 1 (section
 * 特征映射, eq. elu, alpha = 1),
 *
 *     V'_i = phi(Q_i)^T S_i / phi(Q_i)^T Z_i,                       (eq. output)
 *     S_i  = sum_{j<=i} phi(K_j) V_j^T,   Z_i = sum_{j<=i} phi(K_j)   (section 三)
 *
 * in the causal case (diagonal included, eq. mask) and with full sums in the
 * non-causal case (section 二, eq. linear).  No scaling is applied to Q or K.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Tensors are contiguous, row-major, in DEVICE memory of the current CUDA
 *   device: Q, K are [B][H][N][D]; V, Out, dOut are [B][H][N][M]; states S are
 *   [B][H][D][M] and Z are [B][H][D], always fp32.  Every non-empty tensor
 *   pointer must be 16-byte aligned.
 * - dtype: LA_DTYPE_F32 (fp32 storage) or LA_DTYPE_BF16 (bf16 storage).
 *   Outputs have the input dtype, except decode `out` and all states (fp32).
 *   All accumulation is fp32.
 * - Supported head sizes: D, M in {32, 64, 128}.  B, H, N >= 0; a call with
 *   B*H*N == 0 does no work and succeeds.  B*H*N*max(D,M) < 2^40.
 * - `stream` is a cudaStream_t (NULL = legacy default stream).  Every call is
 *   asynchronous on that stream; arguments are validated on the host before
 *   anything is enqueued, and an invalid call enqueues nothing.
 * - Ownership: the caller owns every buffer it passes.  The library never
 *   frees caller memory.  Per-call scratch (span states, gradient rows) is
 *   taken stream-ordered from a library-owned CUDA memory pool of the current
 *   device and given back on the same stream; la_workspace_bytes gives its
 *   size for each call (the gated scan's and the paged cache's calls have
 *   functions of their own).
 * - Errors: a status code; no exception or abort crosses the ABI.  On error,
 *   la_last_error_message() gives a one-line reason (per host thread).
 *
 * Library scratch is stream-ordered, so calls on different streams may run
 * concurrently.
 */
#ifndef LINATTN_H
#define LINATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    LA_OK = 0,
    LA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, negative size, overflow */
    LA_ERR_UNSUPPORTED = 2, /* D or M not in {32, 64, 128}, unknown dtype */
    LA_ERR_CUDA = 3,        /* a CUDA runtime call failed (message has details) */
    LA_ERR_TIMEOUT = 4,     /* a bounded device-side wait gave up (see la_check_device_status) */
    LA_ERR_BAD_INDEX = 5    /* a length, page or slot in device memory was out of range (likewise) */
} la_status;

typedef enum { LA_DTYPE_F32 = 0, LA_DTYPE_BF16 = 1 } la_dtype;

/*
 * Causal forward V' = phi(Q) S_i / phi(Q) Z_i ("Transformers are RNNs",
 * section 三, eq. mask and eq. output).
 *   Q, K    [B][H][N][D] dtype          (read)
 *   V       [B][H][N][M] dtype          (read)
 *   Out     [B][H][N][M] dtype          (written)
 *   S_init  [B][H][D][M] fp32, nullable (read)  state before token 0 (0 if NULL)
 *   Z_init  [B][H][D]    fp32, nullable (read)  must be NULL iff S_init is NULL
 *   S_final [B][H][D][M] fp32, nullable (written) state after token N-1
 *   Z_final [B][H][D]    fp32, nullable (written) must be NULL iff S_final is NULL
 *   Den     [B][H][N]    fp32, nullable (written) the normaliser phi(Q_i).Z_i
 *           of every token (the denominator of eq. output), for the backward
 *   Ckpt    fp32, nullable (written) la_causal_ckpt_floats(B, H, N, D, M)
 *           words: the state (S_i, Z_i) of every head before every 1024th
 *           token, for the backward (written by the bf16 D = M = 64 path;
 *           the other paths leave it untouched)
 * With S_init/Z_init a sequence can be processed in pieces; S_final/Z_final
 * hand a prefill's state to la_decode_step (section 三（二）: the state phi(K)V^T
 * is kept as an internal RNN state).  Out, Den and Ckpt may not alias any input.
 */
la_status la_forward_causal(const void* Q, const void* K, const void* V, void* Out,
                            int B, int H, int N, int D, int M, la_dtype dtype,
                            const float* S_init, const float* Z_init,
                            float* S_final, float* Z_final, float* Den, float* Ckpt,
                            void* stream);

/*
 * Size in fp32 words of the optional state checkpoints of la_forward_causal /
 * la_backward_causal: B * H * ceil(ceil(N / 128) / 8) * (D * M + D), or 0 for
 * non-positive sizes.  Pure arithmetic; no device call.
 */
size_t la_causal_ckpt_floats(int B, int H, int N, int D, int M);

/*
 * Causal backward of L(Out) given dOut = dL/dOut: the numerator gradients of
 * section 三（一）4 (eqs. gq-gv: a prefix state for phi(Q), a suffix state for
 * phi(K) and V), the denominator by the quotient rule, then the chain rule
 * through phi.
 *   Q, K [B][H][N][D]; V, dOut [B][H][N][M] dtype        (read)
 *   Out  [B][H][N][M] dtype, nullable                    (read) the forward's
 *        output; when NULL it is recomputed.
 *   Den  [B][H][N] fp32, nullable                        (read) the forward's
 *        normaliser per token (la_forward_causal's Den, from the same inputs);
 *        the bf16 D = M = 64 path then skips recomputing it, the other paths
 *        ignore it.  The results agree within the bf16 tolerance either way.
 *   Ckpt nullable (read) la_forward_causal's checkpoints from the same inputs
 *        and no S_init; the bf16 D = M = 64 path then starts each part of a
 *        sequence from the nearest one instead of re-reading K and V from the
 *        head's start; the other paths ignore it.
 *   dQ, dK [B][H][N][D]; dV [B][H][N][M] dtype           (written)
 * Outputs may not alias inputs or each other.
 */
la_status la_backward_causal(const void* Q, const void* K, const void* V, const void* Out,
                             const void* dOut, void* dQ, void* dK, void* dV,
                             int B, int H, int N, int D, int M, la_dtype dtype,
                             const float* Den, const float* Ckpt, void* stream);

/*
 * Non-causal forward V' = phi(Q)(phi(K)^T V) / phi(Q) sum_j phi(K_j)
 * ("Transformers are RNNs", section 二, eq. linear and the matrix form
 * (phi(Q)phi(K)^T)V = phi(Q)(phi(K)^T V)).
 *   Q, K [B][H][N][D]; V [B][H][N][M] dtype (read);  Out [B][H][N][M] dtype (written).
 * The call's kernels run in `stream` after the caller's earlier work there.
 * On the fp32 D = M = 64 path the read-out kernel is launched as a
 * programmatic dependent of the state kernel (it starts under that kernel's
 * tail and waits for its partials itself); the chain stays inside the call,
 * and a CUDA graph that captures the call keeps it.
 */
la_status la_forward_noncausal(const void* Q, const void* K, const void* V, void* Out,
                               int B, int H, int N, int D, int M, la_dtype dtype,
                               void* stream);

/*
 * Non-causal backward: the gradient of L(Out) given dOut = dL/dOut for
 * la_forward_noncausal's output.  The numerator gradients of "Transformers
 * are RNNs" section 三（一）4 (eqs. gq-gv) with the prefix state of phi(Q) and
 * the suffix state of phi(K) and V both summed over every token (the
 * unmasked sums of section 二, eq. linear), the denominator by the quotient
 * rule, then the chain rule through phi:
 *   gn_i = dOut_i / den_i, gd_i = -(dOut_i . Out_i) / den_i, den_i = phi(Q_i).Z
 *   dphi(Q_i) = S gn_i + Z gd_i;  R = sum_i phi(Q_i) gn_i^T, r = sum_i phi(Q_i) gd_i
 *   dphi(K_j) = R V_j + r;  dV_j = R^T phi(K_j)
 *   Q, K [B][H][N][D]; V, dOut [B][H][N][M] dtype   (read)
 *   Out  [B][H][N][M] dtype, nullable               (read) the forward's output;
 *        recomputed when NULL
 *   dQ, dK [B][H][N][D]; dV [B][H][N][M] dtype      (written)
 * Outputs may not alias inputs or each other.  On the fp32 D = M = 64 path
 * the call's three kernels are chained by programmatic dependent launch, as
 * in la_forward_noncausal; ordering with the caller's work is unchanged.
 */
la_status la_backward_noncausal(const void* Q, const void* K, const void* V, const void* Out,
                                const void* dOut, void* dQ, void* dK, void* dV,
                                int B, int H, int N, int D, int M, la_dtype dtype, void* stream);

/*
 * One recurrent decode step for B*H independent heads ("Transformers are
 * RNNs" section 四, the RNN form; "Transformer与RNN的深层联结" section 2,
 * RNN-mode inference): first S += phi(k) v^T and Z += phi(k), then
 * out = phi(q)^T S / phi(q)^T Z.
 *   q, k [B][H][D]; v [B][H][M] dtype     (read)
 *   S [B][H][D][M], Z [B][H][D] fp32      (read and updated in place)
 *   out [B][H][M] fp32                    (written)
 * The caller owns S and Z (a session's state can be saved, restored or moved
 * by copying them).  out may not alias S, Z or the inputs.
 */
la_status la_decode_step(const void* q, const void* k, const void* v, float* S, float* Z,
                         float* out, int B, int H, int D, int M, la_dtype dtype, void* stream);

/*
 * Attention with the degree-2 polynomial similarity sim(q, k) = (q^T k)^2 in
 * its linear form ("【论文解读】Transformers are RNNs", section 二 (3): the
 * explicit feature map phi(x) = (x_a x_b), C = D^2 features, cost O(N D^2 M)):
 *     V'_i = phi(Q_i)^T S / phi(Q_i)^T Z,  S = sum_j phi(K_j) V_j^T,  Z = sum_j phi(K_j)
 * over j <= i when causal != 0 (section 三), else over all j.  Raw Q and K
 * (no elu).  Q, K [B][H][N][D]; V [B][H][N][M] dtype (read); Out [B][H][N][M]
 * dtype (written).  Built for D = 32 and M in {32, 64} (LA_ERR_UNSUPPORTED
 * otherwise).  A row whose query is orthogonal to every key it sees has a zero
 * denominator and no defined output.
 */
la_status la_forward_poly2(const void* Q, const void* K, const void* V, void* Out, int B, int H,
                           int N, int D, int M, la_dtype dtype, int causal, void* stream);

/*
 * Linear attention with decay ("retention"), as "Transformer and Variants"
 * (by-xin.github.io) writes it: section 1.3.2 (linear attention as an RNN
 * without the reflection term, no softmax and no normaliser) and section
 * 1.3.4 (RetNet: a decay gamma per head; gated retention: a decay gamma_t per
 * token), with the state in the S = sum k v^T convention (the page's H
 * transposed):
 *     S_t = gamma_t S_{t-1} + k_t v_t^T,   Out_t = S_t^T q_t
 * Raw Q and K (no feature map).
 *   Q, K [B][H][N][D]; V [B][H][N][M] dtype (read);  Out [B][H][N][M] dtype (written)
 *   gamma_head [H] fp32, nullable: RetNet's decay of each head
 *   gates      [B][H][N] fp32, nullable: gated retention's decay of every token
 *              (the page's sigmoid(W_gamma x_t), computed by the caller)
 *   neither: decay 1 (the unnormalised form); both: LA_ERR_INVALID_ARG.
 *   Decays lie in (0, 1]; one below 2^-64 acts as 2^-64.
 *   S_init [B][H][D][M] fp32, nullable (read): state before token 0 (0 if NULL)
 *   S_final [B][H][D][M] fp32, nullable (written): state after token N-1
 */
la_status la_forward_retention(const void* Q, const void* K, const void* V, void* Out, int B,
                               int H, int N, int D, int M, la_dtype dtype, const float* gamma_head,
                               const float* gates, const float* S_init, float* S_final,
                               void* stream);

/*
 * One retention decode step for B*H heads: S = gamma S + k v^T, then
 * out = S^T q ("Transformer and Variants" section 1.3.4, RNN form).
 *   q, k [B][H][D]; v [B][H][M] dtype      (read)
 *   gamma_head [H] fp32, nullable; gate [B][H] fp32, nullable (this step's
 *   decay of each head); neither: decay 1
 *   S [B][H][D][M] fp32                    (read and updated in place)
 *   out [B][H][M] fp32                     (written)
 */
la_status la_retention_decode_step(const void* q, const void* k, const void* v,
                                   const float* gamma_head, const float* gate, float* S, float* out,
                                   int B, int H, int D, int M, la_dtype dtype, void* stream);

/*
 * One decode step of standard softmax attention with a KV cache, the baseline
 * the recurrent step is measured against ("Transformer与RNN的深层联结",
 * section 2, standard Transformer inference: the step's k, v are appended to
 * the cache, then out = softmax(q K^T / sqrt(D)) V over every cached position;
 * the scaled dot product of "Transformers are RNNs", section 一, eq. softmax).
 * Its cost grows with the cache; la_decode_step's does not.
 *   q, k [B][H][D]; v [B][H][M] dtype               (read)
 *   K_cache [B][H][T_max][D], V_cache [B][H][T_max][M] dtype
 *           rows 0..T-1 read; row T written with k, v
 *   T       positions already cached, 0 <= T < T_max (same for every head)
 *   out     [B][H][M] fp32                          (written)
 * Needs D == M (in {32, 64, 128}); LA_ERR_UNSUPPORTED otherwise.  Scratch:
 * la_workspace_bytes("la_softmax_decode_step", B, H, T, D, M, ...).
 */
la_status la_softmax_decode_step(const void* q, const void* k, const void* v, void* K_cache,
                                 void* V_cache, int T, int T_max, float* out, int B, int H, int D,
                                 int M, la_dtype dtype, void* stream);

/*
 * Gated linear recurrence, one decay per token and channel (gated retention's
 * gamma_t, "Transformer and Variants" section 1.3.4, with a state of one value
 * per channel): over the rows t of each sequence and every channel c,
 *   LA_GATE_DECAY   h_t = a_t h_{t-1} + x_t                 (a_t the decay itself)
 *   LA_GATE_LOGIT   h_t = s_t h_{t-1} + (1 - s_t) x_t,  s_t = sigmoid(a_t)
 * from h_init (or 0).  Token-major rows, any channel count C >= 1.
 *   A, X  [B][N][C] dtype                       (read)
 *   Out   [B][N][C] dtype                       (written) h_t rounded to dtype
 *   seq_starts [num_seqs + 1] int32, nullable   (read) packed sequences: with it
 *         B must be 1, and rows seq_starts[i] .. seq_starts[i+1] - 1 are sequence
 *         i (non-decreasing, from 0 up; empty sequences allowed).  Rows behind
 *         the last sequence are not written.  Values outside 0 .. N act as if
 *         cut to that range.  NULL: every batch row is a sequence, num_seqs 0.
 *   h_init  [sequences][C] fp32, nullable (read)     state before the first row
 *   h_final [sequences][C] fp32, nullable (written)  state after the last row
 *         (of an empty sequence: h_init, or 0)
 *   Ckpt  fp32, nullable (written) la_gated_scan_ckpt_floats(B, N, C) words
 *         [B][ceil(N / 128)][C] for the backward: entry k holds the state after
 *         row 128 (k + 1) - 1 where a row follows that one; the last entry of
 *         each batch row, and entries after rows of no sequence, hold no state
 * N <= 2^31 - 129, num_seqs < 2^29 - 1 and B * N * C < 2^40.
 * The logit form's s_t and 1 - s_t are each formed without cancellation: the
 * smaller is within (|a_t| + 6) 2^-23 of itself, the other is one less it.
 * Decays lie in [-1, 1]; the state is fp32 throughout.  Rows are summed up in
 * parts, whose products of decays may round to 0: behind an infinite or NaN
 * state, the rows of its channel and sequence are infinite or NaN.  A sequence's
 * rows do not depend on other sequences, whatever values those hold.  Out,
 * h_final and Ckpt may not alias inputs or each other.  Results do not depend on
 * the run: every sum has a fixed order.
 */
typedef enum { LA_GATE_DECAY = 0, LA_GATE_LOGIT = 1 } la_gate_form;
la_status la_forward_gated_scan(const void* A, const void* X, void* Out, int B, int N, int C,
                                la_dtype dtype, la_gate_form form, const int* seq_starts, int num_seqs,
                                const float* h_init, float* h_final, float* Ckpt, void* stream);

/*
 * The same for a padded row axis: with fill 1, rows that belong to no packed sequence are
 * written too, with 0.  (With fill 0 they are left as they are, as by the call above.)
 */
la_status la_forward_gated_scan_padded(const void* A, const void* X, void* Out, int B, int N, int C,
                                       la_dtype dtype, la_gate_form form, const int* seq_starts,
                                       int num_seqs, const float* h_init, float* h_final, float* Ckpt,
                                       int fill, void* stream);

/* Size in fp32 words of the gated scan's checkpoints: B * ceil(N / 128) * C, or
 * 0 for non-positive sizes.  Pure arithmetic; no device call. */
size_t la_gated_scan_ckpt_floats(int B, int N, int C);

/* Scratch bytes that one la_forward_gated_scan (backward == 0) or
 * la_backward_gated_scan call takes from the library pool, with or without
 * checkpoints; SIZE_MAX for sizes that the call refuses.  Pure arithmetic.
 * la_gated_scan_decode_step takes none. */
size_t la_gated_scan_workspace_bytes(int backward, int B, int N, int C, la_dtype dtype, int ckpt_given);

/*
 * Gradient of la_forward_gated_scan: with s_t the decay and g_t the whole
 * gradient at h_t,
 *   g_t = dOut_t + s_{t+1} g_{t+1}   (last row of a sequence: dOut_t + dh_final)
 *   LA_GATE_DECAY   dA_t = g_t h_{t-1},                          dX_t = g_t
 *   LA_GATE_LOGIT   dA_t = s_t (1 - s_t) g_t (h_{t-1} - x_t),    dX_t = (1 - s_t) g_t
 *   dh_init = s_1 g_1 (first row of a sequence; dh_final or 0 for an empty one)
 *   A, X, dOut [B][N][C] dtype                  (read)
 *   dA, dX     [B][N][C] dtype                  (written; rows behind the last
 *              packed sequence are not)
 *   seq_starts, num_seqs, h_init                as given to the forward
 *   dh_final [sequences][C] fp32, nullable (read)    dL/dh_final (0 if NULL)
 *   dh_init  [sequences][C] fp32, nullable (written) dL/dh_init
 *   Ckpt  nullable (read) the forward's checkpoints from the same inputs; the
 *         call computes them itself when NULL
 * The states are recomputed in fp32 from the inputs; the forward's rounded Out
 * is not used.  Outputs may not alias inputs or each other.
 */
la_status la_backward_gated_scan(const void* A, const void* X, const void* dOut, void* dA, void* dX,
                                 int B, int N, int C, la_dtype dtype, la_gate_form form,
                                 const int* seq_starts, int num_seqs, const float* h_init,
                                 const float* dh_final, float* dh_init, const float* Ckpt,
                                 void* stream);

/* The same for a padded row axis: rows of no sequence get 0 in dA (fill 1), dX (2) or both (3). */
la_status la_backward_gated_scan_padded(const void* A, const void* X, const void* dOut, void* dA,
                                        void* dX, int B, int N, int C, la_dtype dtype,
                                        la_gate_form form, const int* seq_starts, int num_seqs,
                                        const float* h_init, const float* dh_final, float* dh_init,
                                        const float* Ckpt, int fill, void* stream);

/*
 * One token of the gated recurrence for B sequences: h is updated in place and
 * out receives it rounded to dtype.
 *   a, x [B][C] dtype (read);  h [B][C] fp32 (read and updated);  out [B][C] dtype (written)
 */
la_status la_gated_scan_decode_step(const void* a, const void* x, float* h, void* out, int B, int C,
                                    la_dtype dtype, la_gate_form form, void* stream);

/*
 * Paged key-value cache, the ragged form of la_softmax_decode_step's cache.
 * Two pools K_pages, V_pages [num_pages][Hkv][page_size][D] hold the positions
 * of many requests; position p of request r is on page
 * block_table[r][p / page_size] at offset p % page_size, and its slot number is
 * page * page_size + offset.  page_size is a power of two up to 1024, and
 * num_pages * page_size < 2^31; a call takes fewer than 2^30 requests.  Lengths,
 * pages and slots are read on the GPU: one that is out of range has its access
 * skipped and is reported by the next la_check_device_status as LA_ERR_BAD_INDEX.
 *
 * la_page_map: the step's bookkeeping, from request lengths.  Request r holds
 * cached_lens[r] positions and gets new_lens[r] more; the pages that these open
 * are taken from free_pages in the order of the requests.
 *   cached_lens, new_lens [R] int32   (read)
 *   free_pages [num_free] int32       (read) page numbers that no request holds
 *   block_table [R][max_pages] int32  (the pages held are read, those opened are
 *              written, the rest is left as it is; a request's positions past
 *              max_pages * page_size are out of range and get slot -1)
 *   slot_map [max_tokens] int32       (written) the slots of the new positions,
 *              request after request; -1 behind the last one, and where a page
 *              is missing (no free page left: its table entry is -1 too)
 *   seq_starts [R + 1] int32          (written) exclusive sums of new_lens: the
 *              rows of each request among the packed new rows
 *   counts [2] int32                  (written) new positions, pages wanted
 * A call changes neither lengths nor free_pages: the caller moves on by
 * counts[1] pages and adds new_lens to cached_lens.  A negative length acts as 0 and
 * is reported, but for a negative cached length without new positions: a row without
 * a request, as in la_paged_decode_step.
 */
la_status la_page_map(const int* cached_lens, const int* new_lens, int R, const int* free_pages,
                      int num_free, int page_size, int num_pages, int* block_table, int max_pages,
                      int* slot_map, int max_tokens, int* seq_starts, int* counts, void* stream);

/*
 * Rows of keys and values into the paged cache.
 *   k, v [T][Hkv][D] dtype (read);  slot_map [T] int32 (read), -1: the row is skipped
 *   K_pages, V_pages [num_pages][Hkv][page_size][D] dtype (the rows' slots written)
 * D in {32, 64, 128}.  A slot that appears twice holds parts of either row.
 */
la_status la_paged_append(const void* k, const void* v, void* K_pages, void* V_pages,
                          const int* slot_map, int T, int Hkv, int D, int num_pages, int page_size,
                          la_dtype dtype, void* stream);

/*
 * One decode step of softmax attention over the paged cache: the step's k, v
 * are appended at position cached_lens[r] of every request (as in
 * la_softmax_decode_step, "Transformer与RNN的深层联结" section 2), then
 *   out = softmax(scale q K^T) V over the request's last `window` positions
 * (all of them if window is 0).  Query head h reads key head h / (Hq / Hkv).
 *   q [R][Hq][D]; k, v [R][Hkv][D] dtype, nullable together   (read)
 *         NULL: nothing is appended and the cached positions alone are attended
 *   K_pages, V_pages [num_pages][Hkv][page_size][D] dtype     (read; the new row written)
 *   block_table [R][max_pages] int32, cached_lens [R] int32   (read)
 *         a negative length marks a row without a request: nothing of it is read
 *         or written
 *   out [R][Hq][D] fp32                                       (written)
 *   lse [R][Hq] fp32, nullable                                (written) log of the
 *         sum of e^(scale q k); joins outputs over parts of a context
 *   scale 0 means 1 / sqrt(D)
 * A request without a position has out 0 and lse -infinity.  An infinite element of
 * a value row makes its column of out infinite or NaN.  Positions whose page is out
 * of range are left out.  D in {32, 64, 128}, Hq a multiple of Hkv.
 * Reads one key and one value row per position and key head for every 16 query heads
 * that share it (once for up to 16, twice for up to 32, and so on);
 * max_pages * page_size < 2^30.  No page may be held by two requests that append
 * to it.  Results do not depend on the run.
 */
la_status la_paged_decode_step(const void* q, const void* k, const void* v, void* K_pages,
                               void* V_pages, const int* block_table, const int* cached_lens, float* out,
                               float* lse, int R, int Hq, int Hkv, int D, int num_pages, int page_size,
                               int max_pages, int window, float scale, la_dtype dtype, void* stream);

/* The same for a padded batch: rows without a request get 0 in out (fill 1), -infinity in
 * lse (2) or both (3). */
la_status la_paged_decode_step_padded(const void* q, const void* k, const void* v, void* K_pages,
                                      void* V_pages, const int* block_table, const int* cached_lens,
                                      float* out, float* lse, int R, int Hq, int Hkv, int D,
                                      int num_pages, int page_size, int max_pages, int window,
                                      float scale, la_dtype dtype, int fill, void* stream);

/* Scratch bytes that one la_paged_decode_step or la_page_map call takes from the
 * library pool (la_paged_append takes none); SIZE_MAX for sizes that the call
 * refuses.  num_sms as in la_workspace_bytes. */
size_t la_paged_decode_workspace_bytes(int R, int Hq, int Hkv, int D, int page_size, int max_pages,
                                       la_dtype dtype, int num_sms);
size_t la_page_map_workspace_bytes(int R);

/*
 * Attention of a chunk of new tokens over the paged cache, the form of
 * la_paged_decode_step for prompts, for parts of long prompts and for several
 * drafted tokens at once.  The rows seq_starts[r] .. seq_starts[r + 1] - 1 of q
 * are request r's new tokens; row i of them stands at position
 * cached_lens[r] + i, and its key and value are in the cache already
 * (la_paged_append with la_page_map's slots; seq_starts is la_page_map's too):
 *   out = softmax(scale q K^T) V over the last `window` positions up to its own
 * (all of them if window is 0).  Query head h reads key head h / (Hq / Hkv).
 *   q [T][Hq][D] dtype                                        (read)
 *   K_pages, V_pages [num_pages][Hkv][page_size][D] dtype     (read)
 *   block_table [R][max_pages] int32, cached_lens [R] int32   (read) positions
 *         BEFORE the new ones; a negative length marks a request that is none:
 *         nothing of its rows is read or written
 *   seq_starts [R + 1] int32                                  (read) not decreasing,
 *         within 0 .. T; if any go back, that is reported and no request is done (all
 *         rows are rows of no request then)
 *   out [T][Hq][D] dtype                                      (written)
 *   lse [T][Hq] fp32, nullable                                (written)
 *   scale 0 means 1 / sqrt(D);  fill: rows of no request get 0 in out (1),
 *         -infinity in lse (2) or both (3); else they are left as they are
 * out may not overlap another tensor.
 * Positions whose page is out of range are left out; a row that sees none has out
 * 0 and lse -infinity.  What lies in the cache behind a row's position, or before
 * its window, does not reach the row, whatever it is.  An infinite element of a value row makes
 * its column of out infinite or NaN.  Weighted values are summed in fp32 before the division by
 * the weights' sum: where the sum of the |values| that a row sees (bf16: of 256 times them)
 * passes the largest fp32 number, its column may be infinite or NaN too.  bf16: the weights are
 * rounded to bf16 (2^-8 of themselves, the outputs' own rounding) for the product with the values;
 * their sum and lse are not (la_paged_decode_step keeps its weights whole and returns fp32, so the
 * same token's outputs of the two calls differ by these roundings).
 * D in {32, 64, 128}, Hq a multiple of Hkv, T * Hq < 2^30, R < 2^20,
 * max_pages * page_size < 2^30.  Results do not depend on the run.
 */
la_status la_paged_prefill(const void* q, const void* K_pages, const void* V_pages, const int* block_table,
                           const int* cached_lens, const int* seq_starts, void* out, float* lse, int T, int R,
                           int Hq, int Hkv, int D, int num_pages, int page_size, int max_pages, int window,
                           float scale, la_dtype dtype, int fill, void* stream);

/* Scratch bytes that one la_paged_prefill call with rows takes from the library pool, whatever its
 * sizes: partial sums of two cut tiles for every block.  num_sms as in la_workspace_bytes. */
size_t la_paged_prefill_workspace_bytes(int D, la_dtype dtype, int num_sms);

/*
 * Rotary positions: pair i of the first `rot` elements of every query and key head,
 * standing at position p, turns by the angle p theta_i,
 *   (y0, y1) = magnitude (x0 cos - x1 sin, x0 sin + x1 cos);
 * LA_ROTARY_HALF pairs elements i and i + rot / 2, LA_ROTARY_INTERLEAVED 2 i and 2 i + 1.
 * Elements from rot on are copied.
 *
 * la_rotary_frequencies (host): the rot / 2 angles a position, as whole numbers of 2^-64
 * turns, which the calls below read from device memory; of these numbers the phase of any
 * position is exact.  They are worked out in double, which puts an angle off by about
 * p theta_i 2^-53 (at most 1.6e-7 at position 2^31).  theta_i = base^(-2 i / rot) (base >= 1), and for contexts `factor`
 * (>= 1) times longer than trained on
 *   LA_ROTARY_LINEAR    theta_i / factor
 *   LA_ROTARY_BASE      base factor^(rot / (rot - 2)) in place of base
 *   LA_ROTARY_BY_PARTS  theta_i (g + (1 - g) / factor), where g goes from 0 to 1 as the turns
 *                       of original_len positions, original_len theta_i / 2 pi, go from
 *                       beta_slow to beta_fast
 * *magnitude is 0.1 ln(factor) + 1 for the last, else 1.  rot is even, from 2 to 128.
 *
 * la_forward_rotary, la_backward_rotary: queries and keys of one call; the backward turns
 * the upstream gradients by the opposite angles.
 *   q, k [B][Hq][N][D], [B][Hk][N][D] dtype (read), q_out, k_out (written); with Hk = 0
 *         the keys may be NULL, with Hq = 0 the queries
 *   strides  host, nullable: per tensor, in the arguments' order, the distances in elements
 *         between batch rows, tokens and heads (elements of a head are adjacent); NULL:
 *         contiguous as above.  Tensors need their element's alignment only; where all
 *         are 16-byte aligned (so are their strides) and rot is a multiple of 32 bytes (16 for
 *         pairs of neighbours), rows move in 16-byte pieces, else in pieces of two elements
 *         or one
 *   positions int32, device, [N] for all batch rows (position_rows 1) or [B][N]
 *         (position_rows B); a negative one marks a row without a token.  NULL
 *         (position_rows 0): first_position, first_position + 1, ...; with B * N = 0 the
 *         array has no element, and may be NULL beside any of these position_rows
 *   fill  rows without a token get 0 in q_out (1), k_out (2) or both (3); else they are
 *         left as they are
 * An output may be its own input (the same address and strides) and may not overlap
 * another tensor.  B * N < 2^30.
 */
typedef enum { LA_ROTARY_HALF = 0, LA_ROTARY_INTERLEAVED = 1 } la_rotary_layout;
typedef enum { LA_ROTARY_UNSCALED = 0, LA_ROTARY_LINEAR = 1, LA_ROTARY_BASE = 2, LA_ROTARY_BY_PARTS = 3 } la_rotary_scaling;

la_status la_rotary_frequencies(int rot, double base, la_rotary_scaling scaling, double factor, double original_len,
                                double beta_fast, double beta_slow, uint64_t* freqs, float* magnitude);
la_status la_forward_rotary(const void* q, const void* k, void* q_out, void* k_out, int B, int N, int Hq, int Hk,
                            int D, const int64_t* strides, const int* positions, int position_rows,
                            int first_position, const uint64_t* freqs, int rot, float magnitude,
                            la_rotary_layout layout, la_dtype dtype, int fill, void* stream);
la_status la_backward_rotary(const void* dq_out, const void* dk_out, void* dq, void* dk, int B, int N, int Hq, int Hk,
                             int D, const int64_t* strides, const int* positions, int position_rows,
                             int first_position, const uint64_t* freqs, int rot, float magnitude,
                             la_rotary_layout layout, la_dtype dtype, int fill, void* stream);

/*
 * The same with a norm of every head before the rotation, in one pass:
 *   n = x / sqrt(mean x^2 + eps) * weight,   y = rotary(n)   (not rounded in between)
 *   q_weight, k_weight [D] fp32, nullable (1 then), shared by all heads   (read)
 *   eps > 0
 * The backward reads the forward's inputs and the upstream gradients, and writes dq, dk and
 *   dq_weight, dk_weight [D] fp32, nullable   (written) sums over all tokens and heads, in
 *         fp32 and in an order that does not depend on the run
 * An output row may be one of its own input rows.  Rows without a token add nothing.
 */
la_status la_forward_norm_rotary(const void* q, const void* k, const float* q_weight, const float* k_weight,
                                 void* q_out, void* k_out, int B, int N, int Hq, int Hk, int D,
                                 const int64_t* strides, const int* positions, int position_rows,
                                 int first_position, const uint64_t* freqs, int rot, float magnitude,
                                 la_rotary_layout layout, float eps, la_dtype dtype, int fill, void* stream);
la_status la_backward_norm_rotary(const void* q, const void* k, const void* dq_out, const void* dk_out,
                                  const float* q_weight, const float* k_weight, void* dq, void* dk,
                                  float* dq_weight, float* dk_weight, int B, int N, int Hq, int Hk, int D,
                                  const int64_t* strides, const int* positions, int position_rows,
                                  int first_position, const uint64_t* freqs, int rot, float magnitude,
                                  la_rotary_layout layout, float eps, la_dtype dtype, int fill, void* stream);

/* Scratch bytes that one la_backward_norm_rotary call with weights' gradients takes from the
 * library pool (the other rotary calls take none); SIZE_MAX for sizes that the call refuses.
 * num_sms as in la_workspace_bytes. */
size_t la_norm_rotary_workspace_bytes(int B, int N, int Hq, int Hk, int D, int num_sms);

/*
 * la_forward_noncausal with no device allocation.  The paper has no
 * counterpart: this is a service for callers that may not allocate device
 * memory inside an op -- a host framework that plans all device memory in
 * advance and gives the op only its inputs and outputs, a plugin runtime that
 * forbids allocation, or a latency-critical loop that cannot pay for an
 * allocator call.  Arguments, layouts and results are those of
 * la_forward_noncausal (up to the order of floating-point summation).
 * Its scratch is one fixed 16 MiB file-scope device array per device.  With
 * CUDA's default lazy module loading the array is committed on a device by
 * the first call there (its address lookup loads the library's device code),
 * and it stays until the process exits, so a caller that plans device memory
 * should make that first call before planning; later calls make no
 * cudaMalloc, cudaFree or other allocating call.  Limit: 2 * B * H * (D*M + D) * 4 bytes must fit in 16 MiB (B*H <= 127
 * at D = M = 128, <= 504 at D = M = 64); larger calls return
 * LA_ERR_INVALID_ARG with the sizes in the message.  The first call on a
 * device looks up the array's device address (cudaGetSymbolAddress) with that
 * device current, so make the first call on each device before any stream
 * capture.  Every call on a device shares the one array and leaves its
 * contents behind; calls whose work overlaps on the GPU (e.g. on two streams)
 * race on it and must be serialised by the caller.
 */
la_status la_forward_noncausal_noalloc(const void* Q, const void* K, const void* V, void* Out,
                                       int B, int H, int N, int D, int M, la_dtype dtype,
                                       void* stream);

/*
 * Scratch of one call, for callers that plan device memory.  The pages'
 * interface keeps the state S, Z (and for the backward the suffix state)
 * inside the operation ("Overview of Linear Attention", Algorithm forward /
 * backward; "Transformer与RNN的深层联结" section 2, the decode loop on
 * state_s, state_z); this library keeps the per-range states, flags and
 * gradient rows that its parallel split needs in a library-owned pool, and
 * this function says how many bytes of it one call holds at its peak.
 *   op       the entry point's name: "la_forward_causal", "la_backward_causal",
 *            "la_forward_noncausal", "la_backward_noncausal", "la_decode_step" (0),
 *            "la_softmax_decode_step" (N = the cache position T),
 *            "la_forward_retention", "la_retention_decode_step" (0),
 *            "la_forward_poly2" or
 *            "la_forward_noncausal_noalloc" (0: it uses its fixed array)
 *   B..M, dtype  the call's sizes and dtype (N is ignored for decode)
 *   saved    for "la_backward_causal": an OR of LA_SAVED_OUT, LA_SAVED_DEN and
 *            LA_SAVED_CKPT for the optional inputs the call will pass
 *            (Out == NULL makes the call recompute the forward, which needs more)
 *   num_sms  SM count of the device the call will run on; <= 0 queries the
 *            current device (the only device call this function makes)
 * Returns the bytes (0 when the call takes no scratch), or SIZE_MAX for an
 * unknown op, unsupported sizes or a failed device query, with the reason in
 * la_last_error_message().  Pure arithmetic when num_sms > 0.
 */
#define LA_SAVED_OUT 1u
#define LA_SAVED_DEN 2u
#define LA_SAVED_CKPT 4u
size_t la_workspace_bytes(const char* op, int B, int H, int N, int D, int M, la_dtype dtype,
                          unsigned saved, int num_sms);

/*
 * Highest number of bytes of the library's scratch pool on the current device
 * held at once since the pool was created or last reset; reset != 0 then sets
 * it back to zero (to the bytes held now).  For checking la_workspace_bytes
 * against what calls actually take.  SIZE_MAX if a CUDA call failed.
 */
size_t la_scratch_peak_bytes(int reset);

/*
 * Test hook for the failure path of the real kernels, off unless called: the
 * next library call on this process that launches the tensor-core causal
 * forward or backward, or the gated scan's, has unit `unit` of its work split
 * (of the scan: tile `unit` in the order in which its tiles are taken, over all
 * batch rows and channel blocks) skip its look-back publication (the flag or
 * words that later units of the same head or channels wait for), and
 * gives every look-back wait of that launch `spin_limit` polls (about 0.3 us
 * each) instead of the default.  The units waiting on the missing flag give
 * up, set the look-back bit (0x2) in the device error word, drain their copies
 * in flight, free their tensor memory and end, so the call returns without a
 * hang; its outputs are then undefined, and la_check_device_status reports
 * LA_ERR_TIMEOUT.  The setting is consumed by that one call.  LA_ERR_INVALID_ARG
 * for unit < 0 or spin_limit == 0.
 * la_paged_prefill in bf16: block `unit` gets no queries, and the wait for them gives up
 * after `spin_limit` polls (about 3.4 us each), and with it the block's other waits; it ends
 * the same way with the wait bit (0x1), and rows of other blocks' tiles alone are as ever.
 */
la_status la_debug_withhold_publication(int unit, unsigned spin_limit);

/* Synchronises `stream`, then reads and clears the current device's error
 * word set by bounded device-side waits.  LA_ERR_TIMEOUT if one gave up since
 * the last check, LA_ERR_BAD_INDEX if only an index in device memory was out of
 * range (the paged cache's calls), LA_ERR_CUDA if the stream reported an error, else LA_OK. */
la_status la_check_device_status(void* stream);

/* Launches one block whose two bounded device waits cannot be met -- an
 * mbarrier phase that nothing completes and a flag that nothing sets, each
 * given up after a few thousand polls (milliseconds) -- so that both set their
 * bits in the current device's error word, the word and bits the library's
 * kernels set when a copy, a product or a look-back flag never arrives.  For
 * testing that failure path: the next la_check_device_status(stream) reports
 * LA_ERR_TIMEOUT (code 0x3) and clears the word, and the device stays usable.
 * Asynchronous on `stream` (a cudaStream_t, NULL for the default stream);
 * LA_OK once launched, LA_ERR_CUDA if the launch failed. */
la_status la_selftest_expired_waits(void* stream);

/* Static text of a status code. */
const char* la_status_string(la_status status);

/* One-line reason for the last non-LA_OK status returned on this host thread. */
const char* la_last_error_message(void);

/* Number of kernels this library has launched in this process. */
uint64_t la_kernel_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif /* LINATTN_H */
