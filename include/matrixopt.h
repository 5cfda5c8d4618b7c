/*
 * matrixopt.h -- C ABI of a GB300 (sm_103a) library for the optimizer step one
 * owner GPU executes for full 2D weight matrices: Muon (momentum, quintic
 * Newton-Schulz orthogonalisation, scaled update), the Sign-Muon sign / 1-bit
 * pack / majority-vote update, AdamW on the 1D tail, and the owner planner;
 * and operators of the training step around it that make the gradients:
 * embedding, expert products, distillation from a teacher's top logits, the
 * experts' routing, the rows' way to them and back, the norms around a block;
 * and AdamW over many tensors with states in 32 or 8 bits.
 *
 * Sources of the operations (web pages on matrix optimizers):
 *   "Riassunto Tecnico: MatrixFSDP" (gist.science/it/paper/2607.05895)
 *     §Metodologia 1 -- every 2D matrix has one owner rank holding it whole;
 *       Newton-Schulz runs there with no matrix communication; 1D tensors go
 *       to a separate "tail" owner that keeps AdamW.
 *     §Metodologia 2 "Metadati MatrixShard & Global Planner" -- a planner
 *       assigns owners balancing resident bytes and optimizer work.
 *   "Riepilogo Tecnico: SignMuon" (gist.science/it/paper/2605.16311)
 *     §2 "Meccanismo Principale" / "Flusso Algoritmico" -- per-worker momentum
 *       and NS polar direction U, S = sign(U), 1-bit packing for the
 *       all-gather variant, majority vote sign(sum S), W <- W - eta * vote.
 *
 * Conventions (every call):
 *   - Returns MO_OK (0) or a negative MO_ERR_* code; nothing aborts and no
 *     exception crosses the boundary.  mo_status_string() names a code.
 *   - Device buffers and the stream belong to the caller.  The library never
 *     allocates device memory: calls that need scratch take a caller-provided
 *     workspace whose size the matching *_workspace_bytes() call reports.
 *   - Device calls are asynchronous on `stream` (a cudaStream_t; NULL is the
 *     legacy default stream).  plan_owners and the *_workspace_bytes calls
 *     are host-only.
 *   - Matrices are row-major with a leading dimension `ld` in ELEMENTS
 *     (ld >= cols).  Device base pointers must be 16-byte aligned and
 *     ld * element_size must be a multiple of 16 bytes, else MO_ERR_ALIGNMENT.
 *   - A matrix with rows == 0 or cols == 0 is skipped; n == 0 is a no-op.
 *   - Calls with distinct workspaces may run concurrently from any threads;
 *     two in-flight calls must not share a workspace.
 */
#ifndef MATRIXOPT_H
#define MATRIXOPT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* mo_stream_t;      /* same type as cudaStream_t */

/* status codes */
#define MO_OK               0
#define MO_ERR_INVALID_ARG (-1)   /* null pointer, negative size, ld < cols, M <= 0, ... */
#define MO_ERR_ALIGNMENT   (-2)   /* base not 16-byte aligned or ld*elem % 16 != 0 */
#define MO_ERR_WORKSPACE   (-3)   /* workspace null, misaligned (256 B) or too small */
#define MO_ERR_CUDA        (-4)   /* a CUDA runtime/driver call failed */
#define MO_ERR_TIMEOUT     (-5)   /* a device-side bounded wait gave up (see mo_check_device_status) */
#define MO_ERR_UNSUPPORTED (-6)   /* valid request outside what this build implements */

/* element types */
#define MO_F32  0
#define MO_BF16 1
/* index types (token ids) */
#define MO_I32  2
#define MO_I64  3
/* 8-bit floats: 4 exponent bits, 3 of mantissa, largest 448, NaN and no infinity */
#define MO_E4M3 4

/* Newton-Schulz arithmetic */
#define MO_NS_BF16 0   /* bf16 tensor-core operands (tcgen05), fp32 accumulate and epilogue */
#define MO_NS_FP32 1   /* fp32 throughout (CUDA cores), for reference-grade accuracy */

/* One 2D parameter owned by this GPU.  W, M and G share rows, cols and ld.
 * W: weights (updated in place), M: momentum state (updated in place),
 * G: gradient (read only).  dtypes are MO_F32 or MO_BF16 each. */
typedef struct {
    int64_t rows, cols, ld;
    int32_t w_dtype, m_dtype, g_dtype, reserved;
    void*       W;
    void*       M;
    const void* G;
} mo_matrix;

/* Muon hyper-parameters.  The step is
 *   M <- mu*M + G                          (heavy-ball momentum)
 *   X <- orient(M): M^T when rows > cols   (so m <= n)
 *   X <- X / ||X||_F  (0 stays 0); with spectral_iters = q > 0 instead
 *        X <- X / (||X||_F * sigma_hat), sigma_hat^2 = v^T A v after q power
 *        iterations v <- A v / ||A v|| from v = ones/sqrt(m) on the Gram
 *        matrix A of X/||X||_F (the spectral scale; SignMuon §4 compares it
 *        with the Frobenius scale).  bf16 NS and ns_steps >= 1 only.
 *   repeat ns_steps: A = X X^T; B = b*A + c*A*A; X <- a*X + B*X
 *   O <- orient back(X)
 *   apply_update != 0:  W <- W - lr*weight_decay*W - lr*update_scale*O
 *   apply_update == 0:  out[i] <- O (dtype out_dtype, layout of matrix i)  */
typedef struct {
    float   mu, lr, update_scale, weight_decay;
    int32_t ns_steps;              /* k >= 0 */
    float   a, b, c;               /* quintic coefficients */
    int32_t ns_precision;          /* MO_NS_BF16 or MO_NS_FP32 */
    int32_t apply_update;
    int32_t out_dtype;             /* MO_F32 / MO_BF16, used when apply_update == 0 */
    int32_t spectral_iters;        /* 0: Frobenius scale; q in 1..64: spectral scale */
} mo_muon_cfg;

/* The flat float32 tail updated by decoupled AdamW at step number `step`
 * (>= 1, the caller counts):
 *   m <- beta1*m + (1-beta1)*g ; v <- beta2*v + (1-beta2)*g^2
 *   W <- W - lr*weight_decay*W - lr*(m/(1-beta1^t)) / (sqrt(v/(1-beta2^t)) + eps) */
typedef struct {
    int64_t      numel;
    float*       W;
    const float* g;
    float*       m;
    float*       v;
    float        lr, beta1, beta2, eps, weight_decay;
    int32_t      reserved;
    int64_t      step;
} mo_adamw_tail;

/* Workspace size (bytes) muon_step_batched needs for these matrices and cfg.
 * Host only.  MO_ERR_INVALID_ARG for bad shapes / cfg. */
int mo_workspace_bytes(const mo_matrix* mats, int n, const mo_muon_cfg* cfg,
                       size_t* bytes_out);

/* One Muon step over n matrices owned by this GPU, plus optionally the AdamW
 * tail (tail may be NULL).  out may be NULL when cfg->apply_update != 0; else
 * it is a host array of n device pointers, output i laid out like matrix i
 * (rows x cols, leading dimension ld).  ws must be 256-byte aligned and at
 * least mo_workspace_bytes() long.  Runs the fused momentum + norm kernel,
 * then the Newton-Schulz phases grouped over all n matrices, the update fused
 * into the last phase, then the tail.  Asynchronous on `stream`. */
int muon_step_batched(const mo_matrix* mats, int n, const mo_muon_cfg* cfg,
                      const mo_adamw_tail* tail, void* const* out,
                      void* ws, size_t ws_bytes, mo_stream_t stream);

/* A Sign-Muon worker's step with the sign extraction and 1-bit packing
 * fused into the last Newton-Schulz epilogue (SignMuon §2 "Flusso
 * Algoritmico" steps 1-3): momentum and NS as muon_step_batched, no weight
 * update, and instead of the direction U the packed words of sign(U) are
 * written to words[i] (host array of n device pointers, ceil(rows*cols/32)
 * uint32 each, sign_pack's layout and tie rule).  The sign is taken of U as
 * stored in cfg->out_dtype, so the words equal sign_pack of the output
 * muon_step_batched would write.  bf16 NS only, ns_steps >= 1, and every
 * matrix's cols a multiple of 32 (else MO_ERR_UNSUPPORTED); ws sized by
 * mo_workspace_bytes. */
int muon_step_sign_packed(const mo_matrix* mats, int n, const mo_muon_cfg* cfg,
                          uint32_t* const* words, void* ws, size_t ws_bytes, mo_stream_t stream);

/* The whole Sign-Muon step of one GPU that holds the M workers (SignMuon §2
 * "Flusso Algoritmico" steps 1-4, "Meccanismo Principale" 3): each worker's
 * momentum, NS and fused sign + 1-bit pack as muon_step_sign_packed (mats[i]
 * is worker i, words[i] receives its packed signs), then the majority vote
 * over the M = n packed buffers and W <- W - lr*vote as sign_vote_update.
 * Every worker has the same rows x cols (cols a multiple of 32); W is
 * rows x cols with leading dimension ld (>= cols), MO_F32 or MO_BF16, element
 * alignment; 1 <= M <= 128 non-empty workers (else MO_ERR_INVALID_ARG or
 * MO_ERR_UNSUPPORTED).  Two launches on `stream`: the NS with the fused pack,
 * then the vote.  W and the words equal those of muon_step_sign_packed +
 * sign_vote_update.  ws sized by mo_workspace_bytes. */
int muon_step_sign_vote(const mo_matrix* mats, int n, const mo_muon_cfg* cfg, uint32_t* const* words,
                        void* W, int w_dtype, int64_t ld, float lr, void* ws, size_t ws_bytes,
                        mo_stream_t stream);

/* Workspace size for ns_orthogonalize on these shapes (host only). */
int ns_workspace_bytes(const int64_t* rows, const int64_t* cols, int n,
                       int precision, size_t* bytes_out);

/* Pure Newton-Schulz on n matrices: out[i] = orient back(NS_k(X_i/||X_i||_F)).
 * X, out: host arrays of n device pointers (X[i] of dtype in_dtype, out[i] of
 * out_dtype), both rows[i] x cols[i] with leading dimension ld[i].
 * steps >= 0; precision MO_NS_BF16 or MO_NS_FP32.  X is not modified;
 * out may not alias X. */
int ns_orthogonalize(const void* const* X, void* const* out,
                     const int64_t* rows, const int64_t* cols, const int64_t* ld,
                     int n, int in_dtype, int out_dtype, int steps,
                     float a, float b, float c, int precision,
                     void* ws, size_t ws_bytes, mo_stream_t stream);

/* ns_orthogonalize for ONE matrix (bf16 tensor-core mode) that allocates
 * nothing and takes no workspace.  The pages have no counterpart: this entry
 * point exists for callers that cannot allocate device memory, such as a
 * plugin handed only its input and output buffers by a host framework that
 * owns and accounts for every byte of device memory, or a latency-critical
 * loop where a cudaMalloc would synchronise the device.
 *   - Scratch: a fixed array of MO_NOALLOC_SCRATCH_BYTES (32 MiB) compiled
 *     into the library in device global memory; every GPU that loads the
 *     library holds it until the process exits.
 *   - Size limit: ns_workspace_bytes() for this shape must not exceed
 *     MO_NOALLOC_SCRATCH_BYTES, else MO_ERR_UNSUPPORTED (for example
 *     768 x 3072 and 1024 x 2048 fit, 2048 x 2048 does not).
 *   - The first call on a device looks up the array's device address (once
 *     per device, with that device current); make that first call before any
 *     stream capture.
 *   - Every call shares the one array per device and it keeps the last
 *     call's contents; calls whose work overlaps on the GPU (other streams,
 *     other threads) race and corrupt each other's results.
 *   - No cudaMalloc, cudaFree or other allocating routine is called.
 *   - A run whose bounded device waits expire (about 2 s) leaves `out`
 *     unspecified and still returns MO_OK (the wait happens on the GPU after
 *     the call returned); ns_orthogonalize_noalloc_status reports it.
 *   - The call's small control block is copied from ordinary (pageable)
 *     host memory with cudaMemcpyAsync, so the call may return only once
 *     that copy has been staged: it is not fully asynchronous to the host.
 *   - The looked-up device address is kept for the life of the process;
 *     calls after a cudaDeviceReset on that device are not supported.
 * Arguments as ns_orthogonalize with n = 1 (X, out device pointers). */
#define MO_NOALLOC_SCRATCH_BYTES (32u << 20)
int ns_orthogonalize_noalloc(const void* X, void* out, int64_t rows, int64_t cols, int64_t ld,
                             int in_dtype, int out_dtype, int steps, float a, float b, float c,
                             mo_stream_t stream);

/* Status of the allocation-free runs on the current device: waits for
 * `stream`, then returns MO_ERR_TIMEOUT if a run's bounded device wait gave
 * up since the last check (and clears that record), else MO_OK; MO_ERR_CUDA
 * if the device cannot be queried.  As mo_check_device_status, applied to the
 * fixed scratch; it allocates nothing. */
int ns_orthogonalize_noalloc_status(mo_stream_t stream);

/* Sign extraction and 1-bit packing (SignMuon §2 step 2 and the all-gather
 * variant of step 3).  Element j of the row-major flattening of U (rows x
 * cols, leading dimension ld, dtype MO_F32/MO_BF16) goes to bit (j % 32) of
 * words[j / 32]; the bit is 1 unless U_j < 0 (so +0, -0 and NaN give 1, the
 * sign(0) = +1 rule).  words has ceil(rows*cols/32) uint32 entries; unused
 * bits of the last word are written 0.  No workspace.  Only element alignment
 * is required of U (4 or 2 bytes) and of words (4 bytes), and any ld >= cols. */
int sign_pack(const void* U, int dtype, int64_t rows, int64_t cols, int64_t ld,
              uint32_t* words, mo_stream_t stream);

/* sign_pack for M same-shaped matrices in one launch (the M workers of a
 * Sign-Muon step): U and words are host arrays of M device pointers, each
 * pair laid out as for sign_pack.  1 <= M <= 128. */
int sign_pack_batched(const void* const* U, int M, int dtype, int64_t rows, int64_t cols,
                      int64_t ld, uint32_t* const* words, mo_stream_t stream);

/* Majority vote over M packed sign buffers and the voted update (SignMuon §2
 * "Meccanismo Principale" item 3 and step 4).  words: host array of M device
 * pointers, each ceil(rows*cols/32) words in sign_pack's layout.  For each
 * element, with c of the M workers voting +1, vote = +1 if 2c >= M (ties go
 * to +1) else -1, and W <- W - lr*vote in float32 (one rounding; a bf16 W is
 * rounded to bf16 once).  1 <= M <= 128 (MO_ERR_INVALID_ARG for M <= 0,
 * MO_ERR_UNSUPPORTED above 128).  W needs element alignment only, any
 * ld >= cols; word buffers need 4-byte alignment. */
int sign_vote_update(const uint32_t* const* words, int M, int64_t rows, int64_t cols,
                     void* W, int w_dtype, int64_t ld, float lr, mo_stream_t stream);

/* The optional local polar step on the vote (SignMuon §2 "Flusso
 * Algoritmico" step 5): the voted sign matrix S_bar (+1/-1, majority of the M
 * packed buffers, ties +1) is orthogonalised locally with the quintic
 * Newton-Schulz iteration (bf16 tensor cores, k = steps, X0 = S_bar/||S_bar||_F)
 * and W <- W - lr * NS(S_bar).  W follows the 16-byte rules of
 * muon_step_batched; ws (256-byte aligned) holds S_bar and the NS buffers,
 * sized by sign_vote_polar_workspace_bytes (host only).  1 <= M <= 128. */
int sign_vote_polar_workspace_bytes(int64_t rows, int64_t cols, int64_t ld, size_t* bytes_out);
int sign_vote_polar_update(const uint32_t* const* words, int M, int64_t rows, int64_t cols,
                           void* W, int w_dtype, int64_t ld, float lr, int steps,
                           float a, float b, float c, void* ws, size_t ws_bytes, mo_stream_t stream);

/* The int8 all-reduce variant of the vote (SignMuon §2 step 3 "Variante
 * All-Reduce": an integer-sum all-reduce of the signs, then the local
 * threshold; 8 bits per element, §2 "Efficienza di Comunicazione").
 * sign_int8 writes out[j] = -1 if U_j < 0 else +1 (int8) over the row-major
 * flattening of U (dense, rows*cols bytes; U element-aligned, any ld >= cols).
 * sign_vote_update_int8 takes a host array of M device pointers to such
 * buffers (the pre-reduction payloads of M workers), forms each element's
 * integer sum and applies W <- W - lr*vote with vote = +1 iff sum >= 0 (ties
 * +1), one fp32 rounding, as sign_vote_update.  1 <= M <= 127 (the int8 sum
 * range): MO_ERR_INVALID_ARG for M <= 0, MO_ERR_UNSUPPORTED above. */
int sign_int8(const void* U, int dtype, int64_t rows, int64_t cols, int64_t ld,
              int8_t* out, mo_stream_t stream);
int sign_vote_update_int8(const int8_t* const* signs, int M, int64_t rows, int64_t cols,
                          void* W, int w_dtype, int64_t ld, float lr, mo_stream_t stream);

/* Owner planner (MatrixFSDP §Metodologia 2), host only.  For matrix i,
 *   bytes_i = rows_i*cols_i*2, flops_i = ns_steps*(4 m^2 n + 2 m^3) (m<=n),
 *   cost_i  = w_bytes*bytes_i/sum(bytes) + w_flops*flops_i/sum(flops);
 * matrices in decreasing cost (ties: lower index first) each go to the rank
 * with the least accumulated cost (ties: lower rank).  Sums run in index
 * order in double, so the plan is reproducible bit for bit.
 * owner_out[n] receives ranks; load_out[world] (nullable) the per-rank cost.
 * world <= 0 or a negative size gives MO_ERR_INVALID_ARG. */
int plan_owners(const int64_t* rows, const int64_t* cols, int n, int world, int ns_steps,
                double w_bytes, double w_flops, int32_t* owner_out, double* load_out);

/* ------------------------------------------------------------------------
 * Operators of the training step around the optimizer: they make the
 * gradients that muon_step_batched and the AdamW tail consume.  Matrices are
 * row-major with a leading dimension in elements, as above; element
 * alignment suffices unless an entry says otherwise.  Outputs must not overlap
 * inputs unless an entry says so.  All sums are float32; those on the tensor
 * cores (expert_linear*) truncate within pieces of 768 terms (float32 results)
 * or 4096 terms (bf16 results), whose sums are added rounded to nearest.
 * ------------------------------------------------------------------------ */

/* Embedding lookup: out[i, :] = scale * W[ids[i], :] for i < n, W vocab x dim
 * (float32 or bf16, ldw >= dim), out n x dim (float32 or bf16, ldo >= dim),
 * one rounding.  ids: MO_I32 or MO_I64; an id outside [0, vocab) (padding)
 * gives a row of zeros.  n == 0 or dim == 0 is a no-op; with vocab == 0 every
 * row is zero.  vocab and n below 2^31 (else MO_ERR_UNSUPPORTED). */
int embedding_lookup(const void* W, int w_dtype, int64_t vocab, int64_t dim, int64_t ldw, const void* ids,
                     int id_dtype, int64_t n, float scale, void* out, int out_dtype, int64_t ldo,
                     mo_stream_t stream);

/* The lookup's gradient, dense: dW[v, :] = scale * sum of dY[i, :] over the
 * i with ids[i] == v (zeros for a token that does not occur), or, with
 * accumulate = 1, dW[v, :] += that (rows of absent tokens untouched).  The
 * positions are sorted by token and each row is summed in float32 in a fixed
 * order, so that the result is the same bit for bit on every call; a bf16 dW
 * is rounded once.  Ids outside [0, vocab) contribute nothing.  A contiguous
 * float32 dW is what mo_adamw_tail takes as g.  ws: 256-byte aligned, of
 * embedding_grad_workspace_bytes (host only); its contents need no
 * initialisation. */
int embedding_grad_workspace_bytes(int64_t n, int64_t vocab, int64_t dim, size_t* bytes_out);
int embedding_grad(const void* dY, int dy_dtype, int64_t n, int64_t dim, int64_t ldy, const void* ids, int id_dtype,
                   int64_t vocab, float scale, void* dW, int dw_dtype, int64_t ldw, int accumulate, void* ws,
                   size_t ws_bytes, mo_stream_t stream);

/* Matrix products grouped by expert.  The rows of X and dY are sorted by
 * expert: expert e holds rows offsets[e] .. offsets[e + 1] - 1 (any number,
 * also none); offsets is a DEVICE array of experts + 1 int32, non-decreasing,
 * within [0, rows] (other values give wrong results, never an access out of
 * range).  W holds one n x k matrix for each expert, expert e at
 * W + e * stride_w (elements), ldw >= k, stride_w >= n * ldw (unused with one
 * expert).  bf16 operands on the tensor cores, float32 sums:
 *   expert_linear        Y[r, :]  = X[r, :] W_e^T                  (rows x n)
 *   expert_linear_dgrad  dX[r, :] = dY[r, :] W_e                   (rows x k)
 *   expert_linear_wgrad  dW_e (+)= sum_r dY[r, :]^T X[r, :]        (n x k each)
 * Rows of no expert (before offsets[0], from offsets[experts] on) give rows
 * of zeros; an expert without rows gives dW_e = 0 (unchanged with accumulate
 * = 1).  Outputs are float32 or bf16 (rounded once; accumulation adds before
 * that rounding).  dW_e sits at dW + e * stride_dw: the gradient G of one
 * mo_matrix.  Operand and output bases are 16-byte aligned and leading
 * dimensions and strides multiples of 16 bytes (MO_ERR_ALIGNMENT), n and k
 * any size.  rows < 2^31 - 512, n and k <= 2^20, experts <= 1024
 * (MO_ERR_UNSUPPORTED above).  ws: 256-byte aligned, of
 * expert_linear_workspace_bytes (host only), zero-filled once by the caller
 * before its first use; it serves all three calls, one at a time, and
 * mo_check_device_status reads its error word. */
int expert_linear_workspace_bytes(int64_t rows, int64_t n, int64_t k, int experts, size_t* bytes_out);
int expert_linear(const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t stride_w, const int32_t* offsets,
                  int64_t rows, int64_t n, int64_t k, int experts, void* Y, int y_dtype, int64_t ldy, void* ws,
                  size_t ws_bytes, mo_stream_t stream);
int expert_linear_dgrad(const void* dY, int64_t ldy, const void* W, int64_t ldw, int64_t stride_w,
                        const int32_t* offsets, int64_t rows, int64_t n, int64_t k, int experts, void* dX,
                        int dx_dtype, int64_t ldx, void* ws, size_t ws_bytes, mo_stream_t stream);
int expert_linear_wgrad(const void* dY, int64_t ldy, const void* X, int64_t ldx, const int32_t* offsets,
                        int64_t rows, int64_t n, int64_t k, int experts, void* dW, int dw_dtype, int64_t lddw,
                        int64_t stride_dw, int accumulate, void* ws, size_t ws_bytes, mo_stream_t stream);

/* Distillation from a teacher's top logits.  For each of n rows: student
 * logits s (vocab, float32 or bf16, ldl >= vocab) and `top` teacher entries
 * (ids idx, logits t, each n x top, contiguous; idx int32 or int64, t float32
 * or bf16).  An entry whose id lies outside [0, vocab) is absent.  With T =
 * temperature > 0, p = softmax(t / T) over the present entries and q =
 * softmax(s / T) over the vocabulary,
 *   loss  = w T^2 sum_k p_k (log p_k - log q[idx_k])
 *   d s_j = g w T (q_j - sum of p_k over the k with idx_k == j)
 * where w = row_weight[row] (null: 1) and g = grad_scale.  T^2 keeps the
 * gradient's size independent of T.  Entries with p_k = 0 in float32 (t = -inf,
 * or far enough below the others) add nothing; q of a logit at -inf is 0 (a row of -inf only has q = 0 throughout),
 * and p_k > 0 there makes the loss +inf.  A row with w = 0, or without a present
 * entry above -inf, has loss 0 and gradient 0 whatever its logits hold; NaN
 * elsewhere propagates within its row.
 *   distill_topk_loss       writes loss[n] and stats[n][2] = {max s, sum exp((s - max)/T)}
 *   distill_topk_grad       from the same inputs and stats writes dlogits
 *   distill_topk_loss_grad  both in one call: the second read of the logits
 *                           finds most of them in L2
 * dlogits is n x vocab, float32 or bf16, ldg >= vocab; it may be the logits
 * themselves (same type and ld).  1 <= top <= 1024 (MO_ERR_UNSUPPORTED
 * above), vocab < 2^31 - 1024, T a normal float32.  n == 0 is a no-op. */
typedef struct {
    int64_t n, vocab, ldl;
    int32_t top, logits_dtype, idx_dtype, teacher_dtype;
    float temperature, grad_scale;
    const void*  logits;
    const void*  idx;
    const void*  teacher;
    const float* row_weight;   /* n floats, or null */
} mo_distill;

int distill_topk_loss(const mo_distill* d, float* loss, float* stats, mo_stream_t stream);
int distill_topk_grad(const mo_distill* d, const float* stats, void* dlogits, int g_dtype, int64_t ldg,
                      mo_stream_t stream);
int distill_topk_loss_grad(const mo_distill* d, float* loss, void* dlogits, int g_dtype, int64_t ldg,
                           mo_stream_t stream);

/* Routing of n rows to experts.  logits is n x experts (float32 or bf16,
 * ldl >= experts).  Row r goes to its `top` experts of largest logit, ties to
 * the lowest index; a logit of -inf (an expert that is switched off) or NaN is
 * never chosen.  A row whose mask byte is 0 (padding) or without a logit above
 * -inf goes nowhere, has gates and gradient 0 and no part in the loss; `rows`
 * is the number of the others.  With p = softmax(logits[r, :]):
 *   idx[r, j]    the j-th chosen expert, or -1 (fewer than `top` to choose from)
 *   gates[r, j]  p of it; with renormalise = 1 over the sum of the row's chosen
 *                (the softmax over the chosen logits); 0 where idx is -1
 *   counts[e]    rows sent to expert e; counts[experts] = rows
 *   offsets[e]   the sum of counts below e: what expert_linear takes
 *   pos[r, j]    the place of that choice among the rows sorted by expert, and by r
 *                within one (0 .. offsets[experts] - 1), or -1
 *   order[i]     (null: not wanted) the row r of place i, -1 from offsets[experts]
 *                on: what embedding_lookup takes as ids to gather the sorted rows
 *   loss         (null: not wanted) two floats:
 *     balance = experts sum_e (counts[e] / (top rows)) (sum_r p[r, e] / rows)
 *     z       = sum_r logsumexp(logits[r, :])^2 / rows        (both 0 if rows = 0)
 * idx, gates and pos are n x top and order n * top, contiguous; counts and
 * offsets have experts + 1 entries.  Sums run in float32 in a fixed order: the
 * same bit for bit on every call.  exp(logit - the row's largest) counts as 0
 * below 2^-126.  1 <= experts <= 1024, 1 <= top <= min(32,
 * experts), n * top < 2^31 - 512 (MO_ERR_UNSUPPORTED above).  With n == 0 counts,
 * offsets and loss are still written.  ws: 256-byte aligned, of
 * expert_route_workspace_bytes (host only); needs no initialisation.
 *
 * expert_route_grad writes, from the same logits and mask, and idx and counts,
 *   dlogits = d(sum dgates gates + balance_coef balance + z_coef z) / d logits
 * (counts constant), n x experts, float32 or bf16, ldg >= experts; it may be the
 * logits themselves (same type and ld).  dgates (float32, n x top, contiguous)
 * may be null. */
typedef struct {
    int64_t n, ldl;
    int32_t experts, top, logits_dtype, renormalise;
    const void*    logits;
    const uint8_t* mask;       /* n bytes, or null: every row */
} mo_route;

int expert_route_workspace_bytes(int64_t n, int experts, int top, size_t* bytes_out);
int expert_route(const mo_route* r, int32_t* idx, float* gates, int32_t* pos, int32_t* order, int32_t* offsets,
                 int32_t* counts, float* loss, void* ws, size_t ws_bytes, mo_stream_t stream);
int expert_route_grad(const mo_route* r, const int32_t* idx, const int32_t* counts, const float* dgates,
                      float balance_coef, float z_coef, void* dlogits, int g_dtype, int64_t ldg, mo_stream_t stream);

/* The rows' way to the experts and back.  pos (int32, n x top, contiguous) gives
 * the place of row r's j-th copy among `slots` rows, as expert_route writes it;
 * places outside [0, slots) are absent, the others distinct.
 *   expert_scatter       Xs[pos[r, j], :] = X[r, :]              (rows of no place keep what they held)
 *   expert_combine       Y[r, :] (+)= sum_j gates[r, j] Ys[pos[r, j], :]     (gates null: 1)
 *   expert_combine_grad  dYs[pos[r, j], :] = gates[r, j] dY[r, :] and
 *                        dgates[r, j] = dY[r, :] . Ys[pos[r, j], :]   (0 where absent)
 * expert_combine with gates null is the gradient of expert_scatter; with
 * accumulate = 1 it adds to Y (the residual stream, a gradient) before the one
 * rounding.  X, Y, dY and Xs, Ys, dYs are float32 or bf16, of any alignment and
 * leading dimension >= dim; dYs has the type of Ys and may be Ys itself (same
 * ld).  In expert_combine_grad gates may be null (1), dgates null (not wanted).
 * A row without places gives Y[r, :] = 0 (unchanged with accumulate = 1).
 * Sums are float32 over j ascending, one rounding.  n == 0 or dim == 0 is a no-op
 * (dgates are 0 with dim == 0).
 * 1 <= top <= 32, n * top and slots < 2^31, dim <= 2^24 (MO_ERR_UNSUPPORTED above). */
int expert_scatter(const void* X, int x_dtype, int64_t n, int64_t dim, int64_t ldx, const int32_t* pos, int top,
                   void* Xs, int xs_dtype, int64_t slots, int64_t ldxs, mo_stream_t stream);
int expert_combine(const void* Ys, int ys_dtype, int64_t slots, int64_t ldys, const int32_t* pos, const float* gates,
                   int64_t n, int top, int64_t dim, void* Y, int y_dtype, int64_t ldy, int accumulate,
                   mo_stream_t stream);
int expert_combine_grad(const void* dY, int dy_dtype, int64_t ldy, const void* Ys, int ys_dtype, int64_t slots,
                        int64_t ldys, const int32_t* pos, const float* gates, int64_t n, int top, int64_t dim,
                        void* dYs, int64_t lddys, float* dgates, mo_stream_t stream);

/* The way from one block's output x to the next block's input h, over a
 * residual stream.  With norm(t) = t / sqrt(mean(t^2) + eps) over a row's dim
 * values, and g the row of `gate` for row r, r / rows_per_gate:
 *   y = residual_scale residual + block_scale g * post * norm(x)
 *   h = pre * norm(y)
 * post null: x enters unnormed; gate null: 1; residual null: 0; pre null: h is not
 * written (and may be null); y null: the stream is not stored (h is wanted then).
 * x and h are n x dim of x_dtype (float32 or bf16), residual and y of stream_dtype;
 * post, pre (dim each) and gate (ceil(n / rows_per_gate) x dim, ldgate >= dim;
 * rows_per_gate >= 1) of param_dtype.  y may be the residual (same ld), h may be x
 * (same ld).  h comes from y before y is rounded to its type.
 *
 * block_norm_grad: from x, the y that was written, dy (stream_dtype, or null: 0)
 * and dh (x_dtype; null with pre null), writes with t = dy + the norm's gradient,
 *   dresidual = residual_scale t          (stream_dtype; null: not wanted; may be dy)
 *   dx    (type of x; may be x or dh)
 *   dpost (dim), dgate (as gate, contiguous), dpre (dim): float32, summed over the
 *         rows in float32 in a fixed order; accumulate = 1 adds to them.  Each is
 *         wanted or null; without its parameter it has to be null.
 * p->residual is not read (and may be null) there.  ws: 256-byte aligned, of
 * block_norm_grad_workspace_bytes (host only; `gates` = rows of gate, 0 without
 * one; the same on every call with these sizes), no initialisation.
 * dim <= 8192, n < 2^31 (MO_ERR_UNSUPPORTED above); n == 0 or dim == 0: no rows,
 * dpost and dpre are 0 (unchanged with accumulate = 1).  gate has no rows with
 * n == 0, so that dgate is not written there: a caller who keeps some clears them. */
typedef struct {
    int64_t n, dim, ldx, ldr, rows_per_gate, ldgate;
    int32_t x_dtype, stream_dtype, param_dtype;
    float   eps, residual_scale, block_scale;
    const void* x;
    const void* residual;
    const void* post;
    const void* gate;
    const void* pre;
} mo_block_norm;

int block_norm(const mo_block_norm* p, void* y, int64_t ldy, void* h, int64_t ldh, mo_stream_t stream);
int block_norm_grad_workspace_bytes(int64_t n, int64_t dim, int64_t gates, size_t* bytes_out);
int block_norm_grad(const mo_block_norm* p, const void* y, int64_t ldy, const void* dy, int64_t lddy, const void* dh,
                    int64_t lddh, void* dx, int64_t lddx, void* dresidual, int64_t lddr, float* dpost, float* dgate,
                    float* dpre, int accumulate, void* ws, size_t ws_bytes, mo_stream_t stream);

/* AdamW over many tensors at once: mo_adamw_tail's step for each of `count`
 * tensors (a host array, read before the call returns), with its own lr and
 * weight decay and the gradient g scaled by grad_scale times *grad_mul (a device
 * float, null: 1; a clipping factor, for example).  W and g are float32 or bf16
 * each (W rounded once, to nearest), contiguous, of any alignment.  The states are
 * float32 (state_dtype MO_F32: m, v; the scales unused), or 8 bits (MO_E4M3): for
 * each 256 consecutive values of the tensor
 *   m = m_scale q,  v = (v_scale s)^2       with q and s e4m3 values in m and v
 * and ceil(numel / 256) float32 scales of each; zeros throughout are the zero
 * state.  Then the update of W uses the new m and v in float32, before they are
 * rounded: with a = max |m| over the block, m_scale = a (1 / 448) and
 *   q = round((m (1 / a)) 448),   s = the same of sqrt(v), a positive one at least 2^-9
 * each operation one float32 rounding to nearest (1 / 448, too; beta m + (1 - beta) g
 * without fused products), so that the states are reproducible bit for bit.  A block with a
 * < 2^-126 is stored as 0; one with a value that is not finite as NaN throughout.
 * dither = 0 rounds to the nearest e4m3 value, ties to even.  A decay by less than
 * half a step (1/32 to 1/16 of a value) is lost then; dither = 1 rounds at random
 * instead, up with a probability of the distance from the value below, so that
 * means are kept.  Its random bits are a hash of (seed, step, index of the tensor
 * in the list, index in the tensor modulo 2^32): the same inputs give the same bits.
 * The step number (>= 1) is `step`, or, with step_ptr not null, the device int64
 * there, which a captured graph reads on each replay.
 * What is written must not overlap, nor a gradient overlap it; gradients may overlap
 * each other.  numel == 0 is skipped, numel < 2^40
 * (MO_ERR_UNSUPPORTED above); beta1, beta2 in [0, 1), eps in [0, 2^125]. */
typedef struct {
    int64_t     numel;
    void*       W;
    const void* g;
    void*       m;
    void*       v;
    float*      m_scale;
    float*      v_scale;
    int32_t     w_dtype, g_dtype, state_dtype;
    float       lr, weight_decay;
    int32_t     reserved;
} mo_adamw_tensor;

typedef struct {
    float   beta1, beta2, eps, grad_scale;
    int64_t step;
    const int64_t* step_ptr;
    const float*   grad_mul;
    uint32_t seed;
    int32_t  dither;
} mo_adamw_cfg;

int adamw_step_batched(const mo_adamw_tensor* tensors, int count, const mo_adamw_cfg* cfg, mo_stream_t stream);

/* Synchronises `stream`, reads the device error word in workspace `ws`
 * (written by bounded waits inside the kernels), clears it, and returns
 * MO_OK, MO_ERR_TIMEOUT or MO_ERR_CUDA. */
int mo_check_device_status(void* ws, mo_stream_t stream);

/* Static string naming a status code. */
const char* mo_status_string(int status);

/* Library version, e.g. 0x000100 for 0.1.0. */
int mo_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MATRIXOPT_H */
