/*
 * spense.h - C interface of the Spense hybrid sparse-dense linear layer on
 * AMD Instinct MI355X (gfx950).
 *
 * The layer (SpenseGPT gist.science explainer, Technical Summary 2.A "The
 * Spense Format"): the input dimension K of a weight matrix W[N,K] is split
 * into a contiguous 2:4 semi-structured region and a contiguous dense region,
 * and the input-split form accumulates both products into one output,
 *
 *     Y[M,N] = X'[:, :K_s] . W_sparse^T + X'[:, K_s:] . W_dense^T,
 *
 * where X' = X[:, pi] and pi lists the sparse columns ascending, then the
 * dense columns ascending.  Which columns stay dense (Technical Summary 2.B
 * "Dense Index Selection Strategies"): the last p% of K (SpenseGPT), or any
 * chosen set moved into the dense block by that permutation (SpenseGPT+).
 * 2:4 means at most two nonzeros in every four consecutive weights (Technical
 * Summary 1 "Problem Statement"); here exactly two slots per group are kept,
 * the two with the largest magnitude, the lower position winning ties.
 *
 * General rules for every entry point:
 *   - All arguments are validated on the host before any HIP call or launch;
 *     a rejected call returns SPENSE_EINVAL / SPENSE_EUNSUPPORTED and has no
 *     side effect.
 *   - "device pointer" means memory the HIP runtime can access from the GPU
 *     current at the call (hipMalloc / torch CUDA tensors).  "host pointer" is
 *     ordinary CPU memory.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *   - A size may be zero where its range says so; matrices and lists without
 *     elements may then be NULL.
 *   - Matrices are row-major; leading dimensions are in elements.
 *   - An output may overlap no operand and no other output, unless a call says so.
 *   - A HIP runtime failure returns SPENSE_EHIP; spense_last_hip_error()
 *     then returns the hipError_t value.  Faults inside a kernel surface at the
 *     caller's next synchronisation, as for any HIP launch.
 *   - The library is not thread-safe per handle: at most one spense_linear may
 *     be in flight on a handle at a time (its split-K and gather workspaces
 *     are shared).
 *   - spense_linear, spense_linear_w8a8, spense_linear_w4a4, spense_linear_fp8b,
 *     spense_glu, spense_experts_linear and spense_experts_linear_fp8b may be
 *     captured in a HIP graph once an eager call
 *     on the same handle has sized its workspaces: a call that has to grow them
 *     synchronises the stream and allocates.  Sparse layers (automatic split
 *     counts): a call at the captured batch size, or a larger one that had to
 *     grow them, which sizes them for every batch size up to its own, whatever
 *     split count the planner picks there (spense_linear_splits with a forced
 *     split count sizes them for that call only).  mx4, fp8b and experts' layers: any
 *     call of the same entry point with at least as many rows (see there; the first
 *     with more rows than any before plans every smaller number too, 0.3 to 0.6 us of
 *     the host for each sixteen rows).  The
 *     calls record kernel launches only; the split-K hand-off counters are reset
 *     by the kernels.  Workspaces that a captured call used stay allocated until
 *     spense_free, so its graph may also be replayed after a call that needed
 *     larger ones; not after spense_free.
 */
#ifndef SPENSE_H
#define SPENSE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPENSE_ABI_VERSION 6

/* Element types.  The numbering is fixed. */
typedef enum spense_dtype {
  SPENSE_F32 = 0,      /* IEEE binary32 */
  SPENSE_BF16 = 1,     /* bfloat16 */
  SPENSE_FP8_E4M3 = 2, /* OCP e4m3fn: bias 7, largest finite 448, no infinities */
  SPENSE_MX4 = 3       /* microscaled e2m1: 32 consecutive columns share a power of two (spense_quantize_mx4) */
} spense_dtype;

typedef enum spense_status {
  SPENSE_OK = 0,
  SPENSE_EINVAL = -1,       /* bad argument (null pointer, size, dense set, ...) */
  SPENSE_EUNSUPPORTED = -2, /* valid but unsupported combination of types */
  SPENSE_ENOMEM = -3,       /* device or host allocation failed */
  SPENSE_EHIP = -4,         /* a HIP runtime call failed */
  SPENSE_ESCRATCH = -5      /* spense_linear_noalloc: the call needs more than its fixed scratch */
} spense_status;

typedef struct spense_layer* spense_handle;

typedef struct spense_layer_info {
  int64_t N, K;           /* weight shape */
  int64_t K_s, K_d;       /* sparse / dense region lengths, K_s + K_d = K, K_s % 4 == 0 */
  int32_t wdtype;         /* spense_dtype of the stored weights */
  int32_t gather;         /* 1 when spense_linear gathers activation columns (pi not the identity
                             on a 128-aligned split), 0 when X is read in place */
  int64_t weight_bytes;   /* bytes the method must stream per call: kept values + 2-bit indices
                             + dense block = N*(K_s/2*b + K_s/8 + K_d*b), b = element bytes */
  int64_t device_bytes;   /* bytes of the device-resident packed form, padding included */
  int32_t split;          /* 0: input-split layer (spense_pack); 1: output-split (spense_pack_rows);
                             2: GLU block (spense_pack_glu); 3: mx4 layer (spense_pack_mx4);
                             4: experts' layers (spense_pack_experts); 5: fp8b layer
                             (spense_pack_fp8b); 6: fp8b experts (spense_pack_experts_fp8b) */
  int64_t N_s, N_d;       /* output-split: 2:4 rows / dense rows (input-split: N and 0); for an
                             output-split layer K_s = K when N_s > 0 and K_d = K when N_d > 0.
                             GLU block: N = K = H, N_s / N_d = 2:4 / dense intermediate indices,
                             K_s / K_d those of the down projection.
                             mx4 and fp8b layers, experts' layers: N, K of one expert, K_d = K, N_s = experts,
                             N_d = output columns (N / 2 of a gate/up layer); weight_bytes of all */
} spense_layer_info;

/*
 * spense_pack - choose the 2:4 mask and build the packed layer (once per weight).
 *
 * Defined by Technical Summary 2.A / 2.B of the SpenseGPT explainer: the dense
 * set is either `dense_cols` (SpenseGPT+ style, any columns, order irrelevant)
 * or, when dense_cols is NULL, the last K_d = round(dense_fraction*K) columns
 * (SpenseGPT style, rounding half away from zero).  In every group of four
 * consecutive sparse-region columns (in pi order) the two entries with the
 * largest magnitude are kept, magnitude being the stored bit pattern with the
 * sign bit cleared; the lower in-group position wins ties.
 *
 *   W          device pointer, [N, ldw] elements of `wdtype`; only [N, K] is read.
 *   wdtype     SPENSE_F32, SPENSE_BF16 or SPENSE_FP8_E4M3.
 *   N, K       N >= 1, K >= 1; ldw >= K.
 *   scales     device pointer, [N] float32 per-output-channel dequantisation scales;
 *              required (non-NULL) iff wdtype == SPENSE_FP8_E4M3, must be NULL otherwise.
 *              Y[m,n] is multiplied by scales[n].
 *   dense_cols host pointer to n_dense distinct int32 column indices in [0, K), or NULL.
 *   n_dense    number of entries in dense_cols (ignored when dense_cols is NULL).
 *   dense_fraction  used only when dense_cols is NULL; must lie in [0, 1].
 *   stream     stream the packing kernels run on.
 *   out        receives the new handle.
 *
 * K - K_d must be a multiple of 4 (SPENSE_EINVAL otherwise).  The call returns
 * after the packed form is complete (it synchronises `stream`), so W and
 * scales may be freed or overwritten once it returns.  The handle owns every
 * buffer it holds; release it with spense_free.
 */
int spense_pack(const void* W, int32_t wdtype, int64_t N, int64_t K, int64_t ldw, const float* scales,
                const int32_t* dense_cols, int64_t n_dense, double dense_fraction, void* stream,
                spense_handle* out);

/*
 * spense_pack_rows - build an output-split layer (once per weight).
 *
 * Output-split form (Technical Summary 2.A of the SpenseGPT explainer; the
 * page uses it for the GLU gate and up projections): the output rows are
 * split instead of the input columns.  Rows in the dense row set keep all
 * their weights; every other row is 2:4 along K, in groups of four
 * consecutive columns (natural column order), with the same magnitude rule
 * and tie-break as spense_pack.  The two row classes produce different output
 * columns, so nothing is accumulated across them.  The dense row set is
 * `dense_rows` (any rows, order irrelevant) or, when dense_rows is NULL, the
 * last N_d = round(dense_fraction*N) rows.  Arguments as for spense_pack,
 * with dense_rows / n_dense naming rows in [0, N).
 *
 * wdtype must be SPENSE_BF16 or SPENSE_FP8_E4M3 (SPENSE_EUNSUPPORTED for
 * SPENSE_F32).  K must be a multiple of 4 when any row is sparse
 * (SPENSE_EINVAL otherwise).  spense_linear, spense_linear_splits, spense_info
 * and spense_free accept the handle; both row classes run in one launch.
 * Synchronises `stream` before returning.
 */
int spense_pack_rows(const void* W, int32_t wdtype, int64_t N, int64_t K, int64_t ldw, const float* scales,
                     const int32_t* dense_rows, int64_t n_dense, double dense_fraction, void* stream,
                     spense_handle* out);

/*
 * spense_pack_glu - build a GLU MLP block (once per block).
 *
 * Technical Summary 2.A and 2.B of the SpenseGPT explainer: in a GLU MLP the
 * gate and up projections are output-split and the down projection is
 * input-split, over one dense set D of intermediate indices (rows D of gate
 * and up, columns D of down keep all their weights); permuting the
 * intermediate indices so that D becomes one contiguous block leaves the
 * block's output unchanged.  That permutation rho = [other indices ascending
 * | D ascending] is applied here at pack time, so spense_glu gathers nothing.
 * Gate/up rows outside D are 2:4 along the hidden dimension; down columns
 * outside D are 2:4 in groups of four consecutive indices of rho (same
 * magnitude rule and tie-break as spense_pack).  The gate nonlinearity is
 * SiLU (the pages do not name it; the GLU models they evaluate use it).
 *
 *   W_gu       device pointer, [2I, ld_gu] elements: rows [0, I) the gate
 *              projection, rows [I, 2I) the up projection, each [I, H].
 *   W_down     device pointer, [H, ld_down] elements: the down projection [H, I].
 *   wdtype     SPENSE_BF16 or SPENSE_FP8_E4M3 (SPENSE_EUNSUPPORTED for SPENSE_F32).
 *   H, I       hidden and intermediate sizes; ld_gu >= H, ld_down >= I.
 *   s_gu, s_down  device pointers, [2I] and [H] float32 per-row scales; required
 *              iff wdtype == SPENSE_FP8_E4M3, NULL otherwise.
 *   dense_idx  host pointer to n_dense distinct intermediate indices in [0, I), or
 *              NULL for the last round(dense_fraction*I) indices.
 * I - |D| must be a multiple of 4, and so must H when I - |D| > 0
 * (SPENSE_EINVAL otherwise).  Synchronises `stream` before returning.
 */
int spense_pack_glu(const void* W_gu, const void* W_down, int32_t wdtype, int64_t H, int64_t I, int64_t ld_gu,
                    int64_t ld_down, const float* s_gu, const float* s_down, const int32_t* dense_idx,
                    int64_t n_dense, double dense_fraction, void* stream, spense_handle* out);

/*
 * spense_glu - Y = down(silu(gate(X)) * up(X)), the GLU block forward.
 *
 *   X     device pointer, [M, ldx] bf16, ldx >= H.
 *   A     device pointer, [M, lda] bf16, lda >= I: caller-owned workspace for the
 *         intermediate silu(gate) * up, written in rho order (column j holds
 *         intermediate index rho[j]; rho from spense_info's split layout:
 *         the 2:4 indices ascending, then the dense ones ascending).
 *   Y     device pointer, [M, ldy] elements of ydtype (SPENSE_F32 or SPENSE_BF16), ldy >= H.
 * Two launches on `stream`: gate and up (both row classes in one grid, the
 * SiLU * up product in its epilogue, rounded to bf16 into A), then down.
 * Workspaces grow as for spense_linear.
 */
int spense_glu(spense_handle h, const void* X, int64_t M, int64_t ldx, void* A, int64_t lda, void* Y,
               int32_t ydtype, int64_t ldy, void* stream);

/*
 * spense_score_glu - SpenseGPT+ importance score of every intermediate index of a GLU block.
 *
 * Technical Summary 2.B of the SpenseGPT explainer: each weight scores
 * |W_ij| * sqrt(H_jj), H = X^T X over calibration inputs of its projection,
 * and the scores are aggregated per intermediate index over the gate, up and
 * down projections.  Here (the pages leave the aggregation open) it is the
 * plain sum over the weights attached to index i:
 *   score[i] = sum_j |Wg[i,j]| sqrt(Hx_jj) + sum_j |Wu[i,j]| sqrt(Hx_jj)
 *            + sum_n |Wd[n,i]| sqrt(Ha_ii),
 * |W| the dequantised magnitude (per-row scale included).
 *
 *   W_gu, W_down, wdtype, H, I, ld_gu, ld_down, s_gu, s_down: as for spense_pack_glu
 *              (bf16 or e4m3 weights, the unpruned block).
 *   X_cal      device pointer, [T, ld_x] bf16: calibration inputs of gate and up, ld_x >= H.
 *   A_cal      device pointer, [T, ld_a] bf16: calibration inputs of down (the block's
 *              intermediate activations), ld_a >= I.
 *   score      device pointer, [I] float32 output.
 * Reductions run in a fixed order (bitwise repeatable).  Offline step: it
 * allocates scratch (hipMalloc) and synchronises `stream`.
 */
int spense_score_glu(const void* W_gu, const void* W_down, int32_t wdtype, int64_t H, int64_t I, int64_t ld_gu,
                     int64_t ld_down, const float* s_gu, const float* s_down, const void* X_cal, int64_t T,
                     int64_t ld_x, const void* A_cal, int64_t ld_a, float* score, void* stream);

/*
 * spense_select_dense - the dense set: the k indices with the highest scores.
 *
 *   score      device pointer, [n] float32 (for example from spense_score_glu).
 *   dense_idx  host pointer, [k] int32 output, ascending; ready for spense_pack_glu.
 * Index i is selected iff fewer than k indices j have score[j] > score[i] or
 * score[j] == score[i] with j < i (ties go to the lower index).  0 <= k <= n.
 * Infinite scores take their place in that order; a NaN score has none, and
 * the call then returns SPENSE_EINVAL (dense_idx untouched).  Allocates
 * scratch (hipMalloc) and synchronises `stream`.
 */
int spense_select_dense(const float* score, int64_t n, int64_t k, int32_t* dense_idx, void* stream);

/*
 * spense_linear - Y = X . W_pruned^T (times the per-channel scales), the layer forward.
 *
 * Input-split execution (Technical Summary 2.A): the sparse region runs on the
 * structured-sparse SMFMAC matrix instructions, the dense region on the same
 * instruction with index words that select every position (a dense 16x64
 * block is two such products), both accumulating into the same fp32
 * accumulators; when the dense set is not a 128-aligned tail the activation
 * columns are gathered through pi, inside the layer kernel for small batches
 * or into a handle-owned workspace by a preceding kernel on the same stream.
 * Accumulation is fp32; products of bf16 activations with bf16 or e4m3
 * weights are exact.
 *
 *   h          handle from spense_pack.
 *   X          device pointer, [M, ldx] elements of `xdtype`, ldx >= K.
 *              xdtype must be SPENSE_F32 for fp32 weights and SPENSE_BF16 otherwise.
 *   M          number of activation rows, M >= 1.
 *   Y          device pointer, [M, ldy] elements of `ydtype`, ldy >= N; only [M, N] is written.
 *   ydtype     SPENSE_F32 (fp32 accumulators as they are) or SPENSE_BF16 (round to nearest even).
 *
 * Asynchronous on `stream`.  Deterministic: repeated calls give bitwise equal
 * Y (split-K partial sums are added in a fixed order).  The first call at a
 * larger M than before may synchronise `stream` and allocate a larger split-K
 * or gather workspace (hipMalloc); SPENSE_ENOMEM if that fails.
 */
int spense_linear(spense_handle h, const void* X, int32_t xdtype, int64_t M, int64_t ldx, void* Y, int32_t ydtype,
                  int64_t ldy, void* stream);

/*
 * spense_linear_splits - spense_linear with the split-K factor forced (tuning and tests).
 * splits == 0 picks automatically; otherwise 1 <= splits <= number of 128-column steps.
 */
int spense_linear_splits(spense_handle h, const void* X, int32_t xdtype, int64_t M, int64_t ldx, void* Y,
                         int32_t ydtype, int64_t ldy, int32_t splits, void* stream);

/*
 * spense_linear_noalloc - spense_linear that allocates nothing.
 *
 * For callers that cannot allocate device memory during the call: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments, result and kernels as spense_linear (automatic split
 * count), bitwise equal to it; only the call's workspaces differ: the split-K
 * counters and partials and the gathered activations live in a fixed device
 * array of 32 MiB that the library holds on every GPU it runs on until the
 * process ends (64 KiB of it for counters), instead of the handle's own
 * workspaces.  Its first call on a device looks the array up and clears its
 * counters (a fill kernel on `stream`); every completed call leaves them
 * cleared.  No hipMalloc, hipFree or other allocating routine is called.
 *
 * A call whose workspaces exceed the array returns SPENSE_ESCRATCH before any
 * launch (for example a chosen dense set gathered for a large batch: M * K_p
 * * 2 bytes, K_p = K rounded up per region to 128 columns).  Every call on
 * one GPU shares that GPU's array, so two such calls that overlap in time on
 * one GPU (different streams, or different host threads) race and must be
 * ordered by the caller; calls on one stream are ordered by the stream.
 */
int spense_linear_noalloc(spense_handle h, const void* X, int32_t xdtype, int64_t M, int64_t ldx, void* Y,
                          int32_t ydtype, int64_t ldy, void* stream);

/*
 * spense_quantize_tokens - per-token e4m3 quantisation of bf16 activations.
 *
 * The SpenseGPT explainer runs its layers in FP8 (Technical Summary 4,
 * "Experimental Results"); the SlideSparse explainer quantises activations
 * per token online, ahead of the 2:4 GEMM (Methodology 2.B "Activation
 * Lifting", 2.C).  The scale rule is not given there; this library uses the
 * absmax rule:
 *   sx[m]     = max_k |X[m][k]| / 448 as an fp32 quotient (448 is the largest
 *               e4m3fn value), or 1 for an all-zero row;
 *   Xq[m][k]  = the e4m3fn code nearest to the fp32 quotient X[m][k] / sx[m],
 *               ties to the even code, sign kept (within range by construction).
 *
 *   X    device pointer, [M, ldx] bf16, finite values, ldx >= K.
 *   Xq   device pointer, [M, ldq] e4m3 codes (uint8), ldq >= K; written.
 *   sx   device pointer, [M] float32; written.
 * 1 <= M <= 2^24, K >= 1 (SPENSE_EINVAL otherwise).  Asynchronous on `stream`.
 */
int spense_quantize_tokens(const void* X, int64_t M, int64_t K, int64_t ldx, uint8_t* Xq, int64_t ldq, float* sx,
                           void* stream);

/*
 * spense_linear_w8a8 - Y = sx[m] * s[n] * sum_k Xq[m][k] * Wp[n][k]: the layer
 * with e4m3 weights and per-token e4m3 activations.
 *
 * The activations are quantised as spense_quantize_tokens does; the same pass
 * writes them in the layer's packed column order (the dense-set permutation
 * rides on the quantisation, as the SlideSparse explainer folds its activation
 * re-ordering into per-token quantisation), into the handle's workspace.
 * Products of two e4m3 values are exact in fp32.  The matrix instructions on codes add
 * several of them at a time and drop what lies more than 13 bits below the largest
 * of those, whatever the type of Y; the rest of the sum runs in fp32, in a fixed
 * order (bitwise repeatable).  So the sum may be off by 2^-10 of sum_k |Xq Wp|, besides
 * its fp32 roundings: far less on ordinary inputs, but where large products cancel
 * more than the result's own rounding.  spense_linear on the layer keeps all bits.
 *
 *   h      an input-split layer packed from SPENSE_FP8_E4M3 weights
 *          (SPENSE_EUNSUPPORTED for other weight types and for output-split
 *          layers and GLU blocks), or a layer from spense_pack_fp8b (see there).
 *   X      device pointer, [M, ldx] bf16, finite values, ldx >= K.
 *   Y      device pointer, [M, ldy] of ydtype (SPENSE_F32 or SPENSE_BF16 RNE), ldy >= N.
 *   splits split-K factor as for spense_linear_splits (0: automatic).
 * Grows the handle's workspaces on first use at a larger M (synchronising
 * `stream`); otherwise asynchronous.  One call in flight per handle.
 */
int spense_linear_w8a8(spense_handle h, const void* X, int64_t M, int64_t ldx, void* Y, int32_t ydtype, int64_t ldy,
                       int32_t splits, void* stream);

/*
 * Microscaled 4-bit weights (mx4).
 *
 * An mx4 matrix of M rows and K columns is
 *   codes   [M, ldc] bytes, ldc >= ceil(K/2): two e2m1 codes a byte, the even
 *           column in the low half; a code is a sign bit above two exponent
 *           bits and one fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6;
 *   scales  [M, lds] bytes, lds >= ceil(K/32): columns 32b .. 32b+31 of a row
 *           stand for code * 2^(scales[b] - 127); 255 makes them NaN.
 *
 * spense_quantize_mx4 - the mx4 matrix nearest to X.
 *
 * Per block of 32 consecutive columns (the last one may be shorter):
 *   scale = clamp(floor(log2(max |x|)) - 2 + 127, 0, 254), 0 for a block of zeros,
 *   code  = the e2m1 number nearest to x * 2^(127 - scale), ties to the even
 *           code, magnitudes above 6 to 6, the sign kept;
 * a block that holds a NaN or an infinity has scale 255 and codes 0.  Exact:
 * the same bits as the formula in any precision.  The unused half of the last
 * byte of an odd K is 0.
 *
 *   X       device pointer, [M, ldx] of xdtype (SPENSE_F32 or SPENSE_BF16), ldx >= K.
 * 0 <= M <= 2^24, 1 <= K <= 2^20.  Asynchronous on `stream`.
 */
int spense_quantize_mx4(const void* X, int32_t xdtype, int64_t M, int64_t K, int64_t ldx, uint8_t* codes, int64_t ldc,
                        uint8_t* scales, int64_t lds, void* stream);

/*
 * spense_dequantize_mx4 - the numbers an mx4 matrix stands for, into Y [M, ldy] of
 * ydtype (SPENSE_F32 or SPENSE_BF16; exact in both, down to the subnormals; 2^128
 * and more, which only scale bytes 253 and 254 can give, become infinities).
 * Sizes as for spense_quantize_mx4.  Asynchronous on `stream`.
 */
int spense_dequantize_mx4(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t M, int64_t K,
                          void* Y, int32_t ydtype, int64_t ldy, void* stream);

/*
 * spense_pack_mx4 - a linear layer with mx4 weights W[N,K] (once per weight).
 *
 * spense_linear runs it on bf16 activations, Y = X . W^T, with every product
 * exact and the sum in fp32; spense_linear_w4a4 quantises the activations
 * first.  With bf16 activations a weight is taken as bfloat16, which holds every
 * code at scale bytes up to 252 (the largest that spense_quantize_mx4 gives); at
 * 253 and 254 a magnitude of 2^128 or more counts as an infinity.  So it does
 * for mx4 experts.  spense_linear_w4a4 takes all of them as they are.
 * spense_info and spense_free accept the handle;
 * spense_linear_splits with a forced split count and spense_linear_noalloc
 * return SPENSE_EUNSUPPORTED.  Synchronises `stream` before returning.
 */
int spense_pack_mx4(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t N, int64_t K,
                    void* stream, spense_handle* out);

/*
 * spense_linear_w4a4 - Y = mx4(X) . W^T on a layer from spense_pack_mx4.
 *
 * X [M, ldx] bf16 is quantised as spense_quantize_mx4 does, into the handle's
 * workspace; products are exact, the sum runs in fp32 in a fixed order.
 * Y [M, ldy] of ydtype (SPENSE_F32 or SPENSE_BF16).  1 <= M <= 2^24.
 * Workspaces, asynchrony and graph capture as for spense_linear on such a layer:
 * a captured call needs an eager one of the same entry point with M at least its
 * own and, for spense_linear, with X aligned alike and ldx at least its own (rows
 * that do not start at 16 bytes, or a K that is no multiple of 8, are laid out in
 * the workspace first, and so are rows 2^22 or more elements apart).
 */
int spense_linear_w4a4(spense_handle h, const void* X, int64_t M, int64_t ldx, void* Y, int32_t ydtype, int64_t ldy,
                       void* stream);

/*
 * spense_pack_experts - the linear layers of E experts (once per set).
 *
 *   W        device pointer, the experts' matrices one after the other: [E*N, ldw]
 *            bf16, ldw >= K, or mx4 codes [E*N, ldw bytes].
 *   wdtype   SPENSE_BF16 or SPENSE_MX4 (SPENSE_EUNSUPPORTED for the others).
 *   scales   mx4: [E*N, lds] bytes; NULL for bf16.
 *   glu      0, or 1 for gate and up projections in one: N = 2I, rows [0, I) of an
 *            expert the gate, rows [I, 2I) the up projection, and the layer
 *            writes the I columns silu(gate) * up.
 * 1 <= E <= 1024.  Synchronises `stream` before returning.
 */
int spense_pack_experts(const void* W, int32_t wdtype, const uint8_t* scales, int64_t E, int64_t N, int64_t K,
                        int64_t ldw, int64_t lds, int32_t glu, void* stream, spense_handle* out);

/*
 * spense_experts_linear - rows grouped by expert through their expert's layer:
 *
 *   Y[r] = X[rows ? rows[r] : r] . W_e^T   for offsets[e] <= r < offsets[e + 1]
 *
 * (or silu(gate) * up).  Only these rows of Y are written; an expert may have
 * none of them, or all.
 *
 *   X        device pointer, [M, ldx] bf16, ldx >= K, 1 <= M <= 2^24 (M = 0 only with R = 0).
 *   adtype   SPENSE_BF16: the activations as they are; SPENSE_MX4: quantised in the
 *            call (mx4 weights only); SPENSE_FP8_E4M3: the same for fp8b weights
 *            (spense_pack_experts_fp8b; bits of the sums: spense_pack_fp8b).
 *   rows     device pointer, [R] int32 rows of X, or NULL (then M >= R); a row
 *            outside [0, M) is taken as zeros.
 *   offsets  device pointer, [E + 1] int32, ascending from 0 on; values past R count as R.
 *   R        grouped rows that rows and Y have room for, 0 <= R <= 2^24.
 *   Y        device pointer, [R, ldy] of ydtype (SPENSE_F32 or SPENSE_BF16), ldy >= N (I).
 * The sizes of the groups stay on the device.  Deterministic; workspaces,
 * asynchrony and graph capture as for spense_linear (R, M and ldx at most those
 * of the eager call, with the same adtype, rows given or not alike and X aligned
 * alike: rows of X that do not start at 16 bytes, or a K that is no multiple of
 * 8, are laid out in the workspace first, and so are rows far apart or beyond 2
 * GB: the rows that are read, or all of X if picked rows may repeat and it has
 * no more than R).
 */
int spense_experts_linear(spense_handle h, const void* X, int32_t adtype, int64_t M, int64_t ldx, const int32_t* rows,
                          const int32_t* offsets, int64_t R, void* Y, int32_t ydtype, int64_t ldy, void* stream);

/*
 * spense_route - the experts of every token, and the tokens grouped by expert.
 *
 *   logits   device pointer, [T, ldl] of ltype (SPENSE_F32 or SPENSE_BF16), ldl >= E.
 *   k        choices per token, 1 <= k <= E <= 1024; T*k <= 2^24, T may be 0.
 *   ids      [T, k] int32: the experts with the largest logits, largest first,
 *            equal ones lower expert first.  NaN and -inf logits are never
 *            taken; a token with fewer than k others has -1 in the missing places.
 *   weights  [T, k] float32: softmax weights, over the token's choices
 *            (renormalize != 0) or over all its logits; 0 in missing places.
 *            +inf logits share the weight equally.
 *   offsets  [E + 1] int32, rows [T*k] int32, pos [T, k] int32: the pairs (token,
 *            choice) grouped by expert, in token order; row r of expert e,
 *            offsets[e] <= r < offsets[e + 1], is token rows[r], and choice j of
 *            token t is row pos[t, j] (-1: missing).  rows is -1 past offsets[E].
 *   work     spense_route_workspace(T, E, k) bytes (enough for fewer tokens too), 4-byte aligned,
 *            may be NULL if 0.
 * All device pointers.  Deterministic, asynchronous on `stream`, graph-capturable,
 * no state kept: calls with workspaces of their own may overlap.
 */
int64_t spense_route_workspace(int64_t T, int64_t E, int32_t k);
int spense_route(const void* logits, int32_t ltype, int64_t T, int64_t E, int64_t ldl, int32_t k, int32_t renormalize,
                 int32_t* ids, float* weights, int32_t* offsets, int32_t* rows, int32_t* pos, void* work, void* stream);

/*
 * spense_experts_combine - Y[t] = sum_j weights[t, j] * O[pos[t, j]], the
 * experts' outputs weighted and brought back to their tokens.
 *
 *   O        device pointer, [R, ldo] of otype (SPENSE_F32 or SPENSE_BF16), ldo >= N.
 *   pos, weights  device pointers, [T, k] (from spense_route); a pos outside
 *            [0, R) adds nothing.
 *   Y        device pointer, [T, ldy] of ydtype (SPENSE_F32 or SPENSE_BF16), ldy >= N.
 * 0 <= T, R <= 2^24, 1 <= k <= 1024, N >= 1.  Summed in fp32 in the order of j,
 * rounded once.  Asynchronous on `stream`.
 */
int spense_experts_combine(const void* O, int32_t otype, int64_t R, int64_t ldo, const int32_t* pos,
                           const float* weights, int64_t T, int32_t k, int64_t N, void* Y, int32_t ydtype, int64_t ldy,
                           void* stream);

/*
 * Block-scaled 8-bit weights and activations (fp8b).
 *
 * An fp8b matrix of M rows and K columns, its blocks `rows` rows high, is
 *   codes   [M, ldc] bytes, ldc >= K: e4m3fn codes;
 *   scales  [ceil(M / rows), lds] float32, lds >= ceil(K / 128): element (m, k)
 *           stands for code * scales[m / rows][k / 128].
 * Weights have rows = 128, activations rows = 1.
 *
 * spense_quantize_fp8b - the fp8b matrix of X.
 *
 * Per block of rows x 128 (the last ones may be smaller):
 *   scale = max |x| / 448 as an fp32 quotient, 1 where that is 0;
 *   code  = the e4m3fn number nearest to the fp32 quotient x / scale, ties to
 *           the even code, magnitudes above 448 to 448, the sign kept;
 * a block that holds a NaN or an infinity has the scale NaN and codes 0.  Exact:
 * the same bits as the formula.
 *
 *   X       device pointer, [M, ldx] of xdtype (SPENSE_F32 or SPENSE_BF16), ldx >= K.
 *   rows    1 or 128.
 * 0 <= M <= 2^24, 1 <= K <= 2^20.  X, codes and scales may not overlap
 * (SPENSE_EINVAL where two start at the same address).  Asynchronous on `stream`.
 */
int spense_quantize_fp8b(const void* X, int32_t xdtype, int64_t M, int64_t K, int64_t ldx, int32_t rows,
                         uint8_t* codes, int64_t ldc, float* scales, int64_t lds, void* stream);

/*
 * spense_dequantize_fp8b - the numbers an fp8b matrix stands for, into Y [M, ldy]
 * of ydtype (SPENSE_F32 or SPENSE_BF16): the product of code and scale, rounded
 * to fp32 and then, for SPENSE_BF16, to bf16.  Sizes as for
 * spense_quantize_fp8b; Y may overlap neither codes nor scales (SPENSE_EINVAL where it
 * starts at their address).  Asynchronous on `stream`.
 */
int spense_dequantize_fp8b(const uint8_t* codes, int64_t ldc, const float* scales, int64_t lds, int32_t rows,
                           int64_t M, int64_t K, void* Y, int32_t ydtype, int64_t ldy, void* stream);

/*
 * spense_pack_fp8b - a linear layer with fp8b weights W[N,K], blocks of 128 x 128
 * (once per weight).
 *
 *   Y[m, n] = sum_b sx[m][b] * sw[n / 128][b] * sum_(k in b) x[m][k] * w[n][k]
 *
 * over the blocks b of 128 columns.  spense_linear takes bf16 activations as they
 * are (sx = 1), spense_linear_w8a8 (splits = 0) quantises them first as
 * spense_quantize_fp8b with rows = 1 does, into the handle's workspace, and
 * spense_linear_fp8b takes activations that are quantised already.  The product of
 * the two scales is rounded to fp32 and multiplied in with a fused multiply-add,
 * block after block.
 *
 * Bits of the inner sums, here and of experts' layers with fp8b weights:
 *   bf16 activations, either Y, and quantised activations into SPENSE_F32: fp32
 *     sums of exact products;
 *   quantised activations (in the call or before it) into SPENSE_BF16: the matrix
 *     instruction on codes, which adds the products of eight consecutive columns
 *     (8i to 8i + 7) at a time and drops what lies more than 13 bits below the
 *     largest of the eight; the eights are added in fp32.  So an inner sum may be
 *     off by 2^-10 of the largest |x * w| of each eight, besides its fp32
 *     roundings: 2e-5 of the result on normally distributed inputs, but where
 *     large products cancel more than the rounding to bf16, and such a Y is not
 *     the SPENSE_F32 one rounded.  A gate/up layer multiplies sums of these bits.
 * A caller to whom that matters asks for SPENSE_F32.
 *
 * spense_info and spense_free accept the handle; spense_linear_splits with a forced split
 * count and spense_linear_noalloc return SPENSE_EUNSUPPORTED.
 * Synchronises `stream` before returning.
 */
int spense_pack_fp8b(const uint8_t* codes, int64_t ldc, const float* scales, int64_t lds, int64_t N, int64_t K,
                     void* stream, spense_handle* out);

/*
 * spense_linear_fp8b - a layer from spense_pack_fp8b on quantised activations.
 *
 *   codes, scales  device pointers, [M, ldc] e4m3 codes, ldc >= K, and [M, lds]
 *            float32, lds >= ceil(K / 128), for example from spense_quantize_fp8b
 *            or spense_block_norm.  ldc, lds < 2^23 (SPENSE_EUNSUPPORTED).
 *   Y        device pointer, [M, ldy] of ydtype (SPENSE_F32 or SPENSE_BF16, which also
 *            choose the bits of the sums: see spense_pack_fp8b), ldy >= N.
 * 1 <= M <= 2^24.  Deterministic; workspaces, asynchrony and graph capture as for
 * spense_linear on such a layer: a captured call needs an eager one of the same
 * entry point with M at least its own and activations aligned alike with row
 * strides at least its own (rows of codes that do not start at 16 bytes, or a K
 * that is no multiple of 16, and rows of bf16 that do not start at 16 bytes, or a
 * K that is no multiple of 8, are laid out in the workspace first, and so are
 * rows of bf16 2^22 or more elements apart and scales 2^21 or more apart).
 */
int spense_linear_fp8b(spense_handle h, const uint8_t* codes, int64_t ldc, const float* scales, int64_t lds, int64_t M,
                       void* Y, int32_t ydtype, int64_t ldy, void* stream);

/*
 * spense_pack_experts_fp8b - the linear layers of E experts with fp8b weights.
 *
 *   W        device pointer, the experts' matrices one after the other: [E*N, ldw] codes.
 *   scales   device pointer, [E*B, lds] float32, B = ceil(N / 128) blocks of rows
 *            to an expert; with glu 2 ceil(N/2 / 128): the gate's, then the up
 *            projection's, each counted from its own first row.
 *   glu      as for spense_pack_experts.
 * 1 <= E <= 1024.  spense_experts_linear runs them, with adtype SPENSE_BF16, or
 * SPENSE_FP8_E4M3 to quantise the activations in the call (rows = 1), and
 * spense_experts_linear_fp8b.  Synchronises `stream` before returning.
 */
int spense_pack_experts_fp8b(const uint8_t* W, const float* scales, int64_t E, int64_t N, int64_t K, int64_t ldw,
                             int64_t lds, int32_t glu, void* stream, spense_handle* out);

/*
 * spense_experts_linear_fp8b - spense_experts_linear on quantised activations:
 * codes [M, ldc] and scales [M, lds] as for spense_linear_fp8b, for a handle from
 * spense_pack_experts_fp8b.  The other arguments, their ranges, workspaces and
 * graph capture as for spense_experts_linear; bits of the sums by Y's type, see
 * spense_pack_fp8b.
 */
int spense_experts_linear_fp8b(spense_handle h, const uint8_t* codes, int64_t ldc, const float* scales, int64_t lds,
                               int64_t M, const int32_t* rows, const int32_t* offsets, int64_t R, void* Y,
                               int32_t ydtype, int64_t ldy, void* stream);

/*
 * spense_block_norm - the pass over the rows between two blocks of a decoder: the
 * norm after a block, its gate, the scaled residual and the norm before the next.
 *
 *   o[t]  = O[t], or sum_j weights[t, j] O[pos[t, j]] (the experts' outputs, as
 *           spense_experts_combine adds them)
 *   b[t]  = post ? rms(o[t]) * post : o[t]          rms(v) = v / sqrt(mean(v^2) + eps)
 *   r[t]  = scale * residual[t] + gate[t] * b[t]
 *   y[t]  = rms(r[t]) * pre
 *
 * in fp32 throughout (squares that sum to 2^128 or more make an infinite mean, and
 * the normalised row 0); r is rounded once into residual_out, y once into Y, from
 * the unrounded r.
 */
typedef struct spense_norm {
  int64_t T, H;              /* rows and columns: 0 <= T <= 2^24, 1 <= H <= 2^20 */
  const void* O;             /* device pointer, [T, ldo] of otype; with pos [O_rows, ldo] */
  int64_t ldo, O_rows;       /* 0 <= O_rows <= 2^24 */
  const int32_t* pos;        /* device pointers, [T, k], or both NULL; a pos outside [0, O_rows) adds nothing */
  const float* weights;
  const void* post;          /* device pointer, [H] of wtype, or NULL: no norm after the block */
  const void* pre;           /* device pointer, [H] of wtype, or NULL: ones */
  const void* gate;          /* device pointer, [T, ldg] of gtype, or NULL: ones */
  int64_t ldg;               /* 0: one row of gates for all */
  const void* residual;      /* device pointer, [T, ldr] of rtype, or NULL: zeros */
  int64_t ldr;
  void* residual_out;        /* device pointer, [T, ldro] of rtype, may be residual itself (ldro == ldr); or NULL */
  int64_t ldro;
  void* Y;                   /* device pointer, [T, ldy] of ytype, or NULL; not both Y and residual_out NULL */
  int64_t ldy;
  float* yscales;            /* device pointer, [T, lds], with ytype SPENSE_FP8_E4M3: Y holds the codes and this
                                the scales of spense_quantize_fp8b (rows = 1) of y; NULL for other types */
  int64_t lds;
  int32_t k;                 /* with pos: 1 <= k <= 1024 */
  int32_t otype, wtype, gtype, rtype; /* SPENSE_F32 or SPENSE_BF16 */
  int32_t ytype;             /* SPENSE_F32, SPENSE_BF16 or SPENSE_FP8_E4M3 */
  float scale, eps;          /* finite scale; finite eps >= 2^-126 */
} spense_norm;

/*
 * One launch to 2^20 rows, asynchronous on `stream`, graph-capturable, no state
 * kept.  Besides residual_out as residual, no output may overlap an input or
 * another output (SPENSE_EINVAL where they start at the same address).
 * Types of operands that are NULL are ignored.  Deterministic.
 */
int spense_block_norm(const spense_norm* n, void* stream);

/* spense_info - sizes of a packed layer (host-side, no synchronisation). */
int spense_info(spense_handle h, spense_layer_info* info);

/*
 * spense_export - write the packed layer in its canonical form (for bit-exact checks).
 *
 *   vals   device pointer, [N, K_s/2] elements of wdtype: the two kept values of each
 *          group, lower position first.
 *   meta   device pointer, [N, ceil(K_s/32)] uint32: group g's nibble (i0 | i1 << 2),
 *          i0 < i1 its kept in-group positions, sits at bits 4*(g%8) of word g/8;
 *          unused nibbles are 0.
 *   mask   device pointer, [N, K_s] uint8: 1 on kept slots (columns in pi order).
 *   dense  device pointer, [N, K_d] elements of wdtype: W[:, pi[K_s:]].
 *   pi     host pointer, [K] int32 column order.
 * Any pointer may be NULL to skip that part.  Synchronises `stream` before returning.
 */
int spense_export(spense_handle h, void* vals, uint32_t* meta, uint8_t* mask, void* dense, int32_t* pi,
                  void* stream);

/*
 * spense_export_rows - canonical form of an output-split layer (for bit-exact checks).
 *
 *   vals   device pointer, [N_s, K/2]: kept values of the 2:4 rows, in rho order.
 *   meta   device pointer, [N_s, ceil(K/32)] uint32, encoded as for spense_export.
 *   mask   device pointer, [N_s, K] uint8, 1 on kept positions.
 *   dense  device pointer, [N_d, K]: the dense rows, in rho order.
 *   rho    host pointer, [N] int32 row order: the 2:4 rows ascending, then the dense rows ascending.
 * Any pointer may be NULL to skip that part.  SPENSE_EINVAL for an input-split
 * handle (and spense_export returns SPENSE_EINVAL for an output-split one).
 * Synchronises `stream` before returning.
 */
int spense_export_rows(spense_handle h, void* vals, uint32_t* meta, uint8_t* mask, void* dense, int32_t* rho,
                       void* stream);

/* spense_free - release the handle and its device buffers (no launch may still use it). */
int spense_free(spense_handle h);

/* Human-readable text for a status code (static storage). */
const char* spense_strerror(int status);

/* hipError_t value of the most recent SPENSE_EHIP or SPENSE_ENOMEM on the calling thread (0 if none); the runtime's own
 * last error has been taken. */
int spense_last_hip_error(void);

/* SPENSE_ABI_VERSION of the loaded library. */
int spense_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SPENSE_H */
