/*
 * mc2_train.h -- the rest of a training step around the grouped experts, from
 * the same library as mc2.h: the gradients of the two ends of the MoE
 * expert-parallel path (mc2_moe_permute, mc2_moe_unpermute), whose middle is
 * mc2_gmm_combine_backward / mc2_gmm_dispatch_backward, and the
 * orthogonalisation of the stacked weight gradients that these leave.
 *
 * The conventions of mc2.h hold for every entry point here: device pointers,
 * buffers and workspaces owned by the caller, arguments checked on the host
 * before anything is enqueued, work ordered on `stream`, data-dependent faults
 * reported in *dev_err with the offending data skipped, 16-byte aligned base
 * pointers, dense row-major matrices. No entry point here allocates,
 * synchronises or records a memset, so each can be captured into a graph.
 */
#ifndef MC2_TRAIN_H_
#define MC2_TRAIN_H_

#include "mc2.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * mc2_moe_unpermute_backward -- gradient of mc2_moe_unpermute,
 *   out[t] = sum_{k < K} probs[t*K + k] * y_full[unpermute_idx[t*K + k]]:
 * with p = unpermute_idx[s] of slot s = t*K + k,
 *   dy[p]     = probs[s] * dout[t]              (one rounding to dtype)
 *   dprobs[s] = sum_{h < H} dout[t][h] * y_full[p][h]        (fp32)
 * Every row of dy has one writer: slot s writes (and dprobs[s] is computed)
 * only where sorted_idx[unpermute_idx[s]] == s, the relation that
 * mc2_moe_permute's two index arrays have. A slot with index -1 is skipped and
 * gets dprobs 0; a slot whose index lies outside [0, min(y_rows, T*K)) or whose
 * row sorted_idx gives to another slot is skipped too, gets dprobs 0 and sets
 * MC2_DEVERR_INDEX. Rows of dy that no slot names are left as they were: with
 * mc2_moe_permute's indices and y_rows == T*K, rows [0, expert_offsets[E]) are
 * written, which are the rows that mc2_gmm_combine_backward reads.
 *
 *   dout (T, H), y_full and dy (y_rows, H): dtype, MC2_BF16 or MC2_F16;
 *   unpermute_idx, sorted_idx (T*K) int32; probs, dprobs (T*K) fp32.
 * dy may be NULL (only dprobs; probs is then not read and may be NULL), and
 * dprobs may be NULL (only dy; y_full is then not read and may be NULL), not
 * both. The outputs must not overlap any input or each other.
 * Constraints: T >= 1, 1 <= K <= 64, H >= 8, H % 8 == 0, T*K < 2^31 - 1,
 * 0 <= y_rows.
 */
int mc2_moe_unpermute_backward(const void* dout, const void* y_full, int64_t y_rows,
                               const int32_t* unpermute_idx, const int32_t* sorted_idx,
                               const float* probs, int64_t T, int K, int64_t H, int dtype,
                               void* dy, float* dprobs, int32_t* dev_err, hipStream_t stream);

/*
 * mc2_moe_permute_backward -- gradient of mc2_moe_permute's row grouping,
 * permuted[unpermute_idx[t*K + k]] = x[t]:
 *   dx[t] = sum_{k < K} dpermuted[unpermute_idx[t*K + k]]
 * accumulated in fp32 in ascending k and rounded once to dtype. Slots with
 * index -1 are skipped (a token with none gets a row of zeros); an index below
 * -1 or >= rows is skipped and sets MC2_DEVERR_INDEX. This is a gather: an
 * index may appear more than once.
 *   dpermuted (rows, H), dx (T, H): dtype, MC2_BF16 or MC2_F16;
 *   unpermute_idx (T*K) int32. dx must not overlap dpermuted, which may be
 *   NULL where rows is 0 (a rank that got no rows: dx is zeros).
 * Constraints: T >= 1, 1 <= K <= 64, H >= 8, H % 8 == 0, T*K < 2^31 - 1,
 * rows >= 0.
 */
int mc2_moe_permute_backward(const void* dpermuted, int64_t rows, const int32_t* unpermute_idx,
                             int64_t T, int K, int64_t H, int dtype, void* dx, int32_t* dev_err,
                             hipStream_t stream);

/*
 * mc2_ns_orthogonalize -- orthogonalises each matrix of a stack (the update of
 * a weight from its gradient or momentum) by Newton-Schulz products. For each
 * of the `batch` matrices G (m, n), with r = min(m, n):
 *   X = G / (|G|_F + eps)
 *   for each step, with its coefficients (a, b, c):
 *     A = X X^T (m <= n) or X^T X (m > n)                          (r, r)
 *     X = a X + (b A + c A A) X       or  a X + X (b A + c A A)
 *   out = scale * X
 * The stacks that mc2_gmm_combine_backward (E_l, I, H) and
 * mc2_gmm_dispatch_backward (E_l, H, I2) leave can be passed as they are.
 *
 *   g (batch, m, n) in_dtype: MC2_F32, MC2_BF16 or MC2_F16; not modified.
 *   steps >= 1, <= 32; coeffs: HOST pointer to 3 * steps floats, (a, b, c) of
 *     each step, every one within [-16, 16]; read before the call returns.
 *   eps >= 0 and scale finite. A matrix of zeros gives zeros.
 *   out (batch, m, n) out_dtype: MC2_BF16 or MC2_F16. out may be g where the
 *     two types have the same size; otherwise they must not overlap.
 *   workspace: caller-owned, 16-byte aligned, at least
 *     mc2_ns_workspace_size(batch, m, n) bytes, no initialisation needed.
 *     Calls that overlap in time must not share one. The size follows from the
 *     arguments alone, not from the device: batch times that of one matrix, or
 *     that of one matrix whatever the batch where one workgroup iterates a
 *     matrix (r padded to 64 at most 128, and at most 64 Ki elements with c
 *     padded to a power of two times 128).
 * Constraints: 1 <= batch <= 65535, 1 <= m, n <= 65536 (any sizes: rows need
 * not be whole 16-byte pieces); mc2_ns_workspace_size gives 0 for sizes outside.
 * batch * ceil(m / 64) * ceil(n / 64) < 2^24 (128 GiB for one copy of the
 * iterate), else MC2_ERR_SHAPE.
 *
 * Precision: the norm is summed in fp64. Products take operands rounded to
 * fp16 (scaled by powers of two) and accumulate in fp32; the iterate itself is
 * held to 22 bits or more until the last step, so that rounding noise in
 * directions whose singular value is near zero is not multiplied by a in every
 * step. With the usual five steps of (3.4445, -4.7750, 2.0315), and before the
 * rounding to out_dtype, the error of the result (2-norm of the difference over
 * that of the result) is 4e-4 to 2.7e-3 for dense matrices of any rank whose
 * singular values differ, r >= 20 (gradients). It is larger where few or equal
 * ones carry the matrix and operand roundings do not average out, since a
 * step magnifies a relative error by up to 5: 9e-3 for identity matrices, and
 * 3.5e-2 at most over the spectra tried (2 or 3 nonzero singular values). More
 * steps magnify it further. |G|_F below 1e-5 eps leaves iterates too small for
 * fp16. Iterates are held in range as long as their entries stay below 16 and
 * the entries of A and b A + c A A below 128 (coefficients whose iterates stay
 * bounded, as those do); beyond, the result is infinite or NaN. A NaN or
 * infinity in G spreads over its own matrix only. The same arguments give the
 * same bits.
 */
size_t mc2_ns_workspace_size(int64_t batch, int64_t m, int64_t n);

int mc2_ns_orthogonalize(const void* g, int64_t batch, int64_t m, int64_t n, int in_dtype,
                         int steps, const float* coeffs, float eps, float scale, int out_dtype,
                         void* out, void* workspace, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MC2_TRAIN_H_ */
