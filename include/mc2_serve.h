/*
 * mc2_serve.h -- operands held in 4 bits (MX4) and the MoE layer for few
 * tokens, from the same library as mc2.h: quantisation and its inverse, the
 * product of two 4-bit operands in the chunk schedule of the rank-chunked
 * GEMM, and a whole mixture-of-experts layer for the tokens of a decoding step.
 *
 * The conventions of mc2.h hold for every entry point here: device pointers,
 * buffers and workspaces owned by the caller, arguments checked on the host
 * before anything is enqueued, work ordered on `stream`, data-dependent faults
 * reported in *dev_err with the offending data skipped, 16-byte aligned base
 * pointers, dense row-major matrices. No entry point here allocates,
 * synchronises or records a memset, so each can be captured into a graph.
 * Outputs must not overlap inputs or each other.
 *
 * MX4 operand (rows, k): every row is cut along k into nb = ceil(k / 32) blocks
 * of 32 values that share a power of two.
 *   codes  (rows, 16 * nb) bytes: two values a byte, the even one in the low
 *          four bits; a value is a sign (bit 3) and one of
 *          0, 0.5, 1, 1.5, 2, 3, 4, 6 (bits 2..0 = 0..7).
 *   scales (rows, nb rounded up to a multiple of 16) bytes: s stands for
 *          2^(s - 127); s = 255 makes its block NaN.
 * A value is its code times its block's power of two. The codes behind the
 * last value of a row and the scales behind its last block are zero in what
 * mc2_mx4_quantize writes; operands that come from elsewhere must hold zeros
 * there too.
 */
#ifndef MC2_SERVE_H_
#define MC2_SERVE_H_

#include "mc2.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Weight type of mc2_moe_tokens beside those of mc2_dtype. */
#define MC2_MX4 5

/* Bytes of codes (16 * nb) and of scales (nb rounded up to 16) in a row of k
 * values; 0 for k < 1 or k > MC2_MX4_MAX_K. */
#define MC2_MX4_MAX_K 1048576
size_t mc2_mx4_row_bytes(int64_t k);
size_t mc2_mx4_scale_bytes(int64_t k);

/*
 * mc2_mx4_quantize -- MX4 form of a stack of matrices. For each block, with m
 * its largest magnitude:
 *   e = floor(log2(m)) - 2, at least -127 (-127 where m is 0);  scale 2^e
 *   code = x / 2^e rounded to nearest, ties to even, 6 where that exceeds 6
 * A block that holds a NaN or an infinity gets the scale 255 and codes 0.
 * Magnitudes in (6, 8) times 2^e are so rounded down to 6 * 2^e: a value is
 * off by at most a quarter of itself, or 2^e / 4 where it is small.
 *
 *   x: in_dtype, MC2_BF16, MC2_F16 or MC2_F32. trans == 0: (batch, rows, k);
 *      trans != 0: (batch, k, rows), so that blocks run along the first axis
 *      (a weight held (k, n), or an operand of a gradient's product).
 *   codes (batch, rows, mc2_mx4_row_bytes(k)), scales (batch, rows,
 *      mc2_mx4_scale_bytes(k)) uint8, fully written.
 * Constraints: 1 <= batch, rows; batch * rows <= 2^36; 1 <= k <= MC2_MX4_MAX_K
 * (any sizes: rows of x need not be whole 16-byte pieces).
 */
int mc2_mx4_quantize(const void* x, int64_t batch, int64_t rows, int64_t k, int trans,
                     int in_dtype, void* codes, void* scales, hipStream_t stream);

/*
 * mc2_mx4_dequantize -- the values that codes and scales stand for, rounded
 * once to out_dtype (exact in MC2_F32 and MC2_BF16 but for magnitudes past the
 * type's largest, which become infinite; MC2_F16 rounds small ones to nearest
 * even and overflows to infinity). out: (batch, rows, k), or (batch, k, rows)
 * where trans != 0: the layout of x in mc2_mx4_quantize. Constraints as there.
 */
int mc2_mx4_dequantize(const void* codes, const void* scales, int64_t batch, int64_t rows,
                       int64_t k, int trans, int out_dtype, void* out, hipStream_t stream);

/*
 * mc2_mx4_mm_rs_local / mc2_mx4_ag_mm_local -- the compute share of
 * MatmulReduceScatter / AllGatherMatmul with both operands in MX4:
 *   out (m, n) = x1 (m, k) @ x2 (n, k)^T + bias
 * accumulated in fp32 and rounded once to out_dtype. x2 is held (n, k), as
 * x2_trans of mc2_mm_rs_local. Gradients are products of the same kind: with
 * x1 = Q(x), x2 = Q(w) in the forward, dx = Q(dy) @ Q(w^T)^T and
 * dw = Q(dy^T) @ Q(x^T)^T, the transposed operands from mc2_mx4_quantize with
 * trans (straight through the quantisation, whose own gradient is 1).
 *
 *   x1, x1_scale: codes and scales of (m, k); x2, x2_scale: of (n, k).
 *   bias NULL or (n) MC2_BF16. out_dtype MC2_BF16, MC2_F16 or MC2_F32.
 *   world_size, rank, comm_turn, ready_flags, flag_counters, epoch: the chunk
 *   schedule and the flags of mc2_mm_rs_local (chunks computed from rank + 1
 *   on) and mc2_ag_mm_local (from rank on; m = W * m_c); world_size in
 *   {1, 2, 4, 8, 16, 32}, m % world_size == 0, 0 <= comm_turn <= m / W.
 * Constraints: m, n >= 1, 1 <= k <= MC2_MX4_MAX_K, n % 8 == 0 (MC2_ERR_ALIGN),
 * n <= 2^20. The same arguments give the same bits; float sums of calls with
 * few rows (no flags) are taken in another order than those with many.
 */
int mc2_mx4_mm_rs_local(const void* x1, const void* x1_scale, const void* x2,
                        const void* x2_scale, int64_t m, int64_t k, int64_t n, int world_size,
                        int rank, const void* bias, int out_dtype, void* out,
                        uint32_t* ready_flags, uint32_t* flag_counters, uint32_t epoch,
                        int comm_turn, hipStream_t stream);

int mc2_mx4_ag_mm_local(const void* x_gathered, const void* x_scale, const void* x2,
                        const void* x2_scale, int64_t m_c, int64_t k, int64_t n, int world_size,
                        int rank, const void* bias, int out_dtype, void* out,
                        uint32_t* ready_flags, uint32_t* flag_counters, uint32_t epoch,
                        int comm_turn, hipStream_t stream);

/*
 * mc2_moe_tokens -- this rank's share of a whole MoE layer for few tokens (a
 * decoding step): what mc2_moe_permute, mc2_gmm_dispatch with SwiGLU,
 * mc2_gmm_combine and mc2_moe_unpermute compute together, in two launches:
 *   a = x[t] @ w1[e];  h = silu(a[:I]) * a[I:];  y = h @ w2[e]
 *   out[t] = sum_{k < K} probs[t*K + k] * y of expert sel[t*K + k]
 * over the slots whose expert is local, ep_rank * E_l <= sel < (ep_rank + 1) *
 * E_l; a token with none gets a row of zeros, and the layer's output is the
 * sum of the ranks' outs. An id outside [0, num_experts) is skipped and sets
 * MC2_DEVERR_EXPERT_ID. An id may appear more than once in a token. Products
 * accumulate in fp32; h, y and the sum over k are fp32, one rounding to bf16.
 * Every expert named by a slot is read once per 32 slots of it, per 16 where
 * T <= 16. Up to some 64 slots an expert the layer takes less time than those
 * four calls, beyond that they do (8 experts of 2048 x 1536 and 768 x 2048 in
 * bf16, K = 8: 64 tokens 64 against 98 us, 128 tokens 118 against 98).
 *
 *   x, out (T, H) bf16; sel (T*K) int32; probs (T*K) fp32.
 *   w_dtype MC2_BF16: w1 (E_l, H, 2I) (gate columns [0, I), up [I, 2I)) and w2
 *     (E_l, I, H), the weights of mc2_gmm_dispatch and mc2_gmm_combine;
 *     w1_scale and w2_scale NULL.
 *   w_dtype MC2_MX4: w1, w1_scale the MX4 form of (E_l, 2I, H) and w2, w2_scale
 *     that of (E_l, H, I): mc2_mx4_quantize with trans of the weights above.
 *     The products are of bf16 activations and exact bf16 values of the codes.
 *   workspace: caller-owned, 16-byte aligned, at least
 *     mc2_moe_tokens_workspace_size(T, K, H, I) bytes, no initialisation
 *     needed. Calls that overlap in time must not share one.
 * Constraints: 1 <= T <= 256, 1 <= K <= 64, T*K <= 4096, H % 8 == 0,
 * I % 8 == 0 (MC2_ERR_ALIGN), 8 <= H, I <= 65536, 1 <= num_experts,
 * 1 <= E_l <= 1024, (ep_rank + 1) * E_l <= num_experts, T*K*H < 2^28,
 * T*K*I < 2^28; mc2_moe_tokens_workspace_size gives 0 for sizes outside. The same
 * arguments give the same bits.
 */
size_t mc2_moe_tokens_workspace_size(int64_t T, int K, int64_t H, int64_t I);

int mc2_moe_tokens(const void* x, const int32_t* sel, const float* probs, int64_t T, int K,
                   int64_t H, int num_experts, int ep_rank, int local_experts, int w_dtype,
                   const void* w1, const void* w1_scale, const void* w2, const void* w2_scale,
                   int64_t I, void* out, void* workspace, size_t ws_bytes, int32_t* dev_err,
                   hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MC2_SERVE_H_ */
