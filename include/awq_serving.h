/*
 * awq_serving.h — C ABI of the operators that serve a packed layer: they stand
 * beside awq_w4a16_gemm when a packed model answers many requests (the pages stop
 * at the packed format; these entries exist for its users).  All activations are
 * fp16, all sums, norm statistics and softmax statistics fp32 or wider.  The
 * conventions of awq.h hold: device pointers and workspace of the caller, calls
 * ordered on `stream`, arguments checked on the host before anything is launched,
 * device-side failures in the workspace's status word (awq_device_status), calls
 * that share a workspace must not overlap (captured graphs that share one neither).
 */
#ifndef AWQ_SERVING_H
#define AWQ_SERVING_H

#include "awq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A packed projection with the low-rank adapter of each token's request
 * beside it:
 *   Y[t][o] = RN16( sum_j X[t][j] W[o][j] + c_a sum_r U[t][r] B_a[o][r] ),
 *   U[t][r] = sum_j X[t][j] A_a[r][j],  W[o][j] = (q - z) scale,  a = adapter[t];
 * a token whose adapter is -1 gets the first sum alone.  Rows may carry their
 * adapters in any order.
 *   X, qweight, qzeros, scales, Y, cfg  as in awq_w4a16_gemm; Y is not X
 *   A        device fp16 [n_adapters, rank, in]
 *   B        device fp16 [n_adapters, out, rank] (an adapter of lower rank is
 *            padded with zeros)
 *   c        device fp32 [n_adapters]: each adapter's scale
 *   adapter  device int32 [T], values in [-1, n_adapters).  Any other value is
 *            an error found on the device: the row is computed without an
 *            adapter and the status word of ws records AWQ_ERR_INVALID_ARG
 *   ws       awq_w4a16_lora_workspace_size() bytes
 * Up to 64 tokens the packed words are streamed and the weights stay
 * (q - z) scale exactly; beyond, they are rounded to fp16 once, as in
 * awq_w4a16_gemm, and c_a U to fp16, for one product on the tensor cores (a token
 * whose largest c_a U is past 65504, or below 2^-12, keeps it in fp32).
 * Requires in % 64 == 0, out % 32 == 0, rank % 8 == 0 and 8 <= rank <= 256,
 * 1 <= n_adapters <= 65536, n_adapters * out < 2^31; X, A, B and Y 16-byte
 * aligned, c and adapter 4-byte aligned. */
awq_status awq_w4a16_lora_gemm(const void *X, int64_t T, int64_t in, int64_t ldx,
                               const int32_t *qweight, const int32_t *qzeros, const void *scales,
                               int64_t out, const awq_config *cfg, const void *A, const void *B,
                               const float *c, int32_t n_adapters, int32_t rank,
                               const int32_t *adapter, void *Y, int64_t ldy, void *ws,
                               size_t ws_bytes, awq_stream_t stream);

/* Workspace bytes of awq_w4a16_lora_gemm; 0 when the arguments are invalid. */
size_t awq_w4a16_lora_workspace_size(int64_t T, int64_t in, int64_t out, int32_t rank,
                                     const awq_config *cfg);

/* A whole mixture-of-experts layer on packed experts, for a few tokens (a
 * decode step or a small batch), in one call: router, choice, gate|up,
 * SwiGLU, down and the weighted sum,
 *   l_te = sum_j X[t][j] router[e][j];  the top_k largest of a row, ties to the
 *   lowest expert;  p = softmax of l_t over all experts, divided by the chosen
 *   ones' sum when renormalize = 1;
 *   H = RN16( silu(x gate_e) (x up_e) );  Y[t] = RN16( sum_k p_k down_e(H) )
 * with every packed weight (q - z) scale unrounded.  An expert's tokens are taken 24
 * at a time (8 at a time up to 8 tokens in all); where that leaves up to four, what
 * H's rounding loses is kept too (22 bits).  H past 65504 is infinite, as its rounding
 * says, and so are its token's outputs.
 *   X       device fp16 [T, hidden], row stride ldx
 *   mask    device uint8 [T] or NULL: rows with 0 (the padding of a captured
 *           step) meet no expert and get ids -1, weights 0 and Y = 0; their X
 *           is not used
 *   router  device fp16 [n_experts, hidden]
 *   gu_*    the experts' gate|up linears packed by awq_quant_pack, gate's
 *           outputs first: qweight [n_experts, hidden, 2 inter/8], qzeros
 *           [n_experts, hidden/g, 2 inter/8], scales fp16 [n_experts, hidden/g, 2 inter]
 *   dn_*    the down linears: qweight [n_experts, inter, hidden/8], qzeros and
 *           scales over inter/g groups
 *   Y       device fp16 [T, hidden] (output), row stride ldy; not X
 *   ids     device int32 [T, top_k] (output), in falling order of their logits
 *   weights device fp32 [T, top_k] (output)
 *   ws      awq_w4a16_moe_workspace_size() bytes
 * Requires 1 <= T <= 64, 1 <= top_k <= min(16, n_experts), n_experts <= 256,
 * hidden and inter multiples of 64 and of cfg->group_size, hidden <= 16384,
 * inter <= 65536; X, router, the packed tensors and Y 16-byte aligned.  The
 * kernel is launched cooperatively (its blocks meet at bounded barriers): a
 * barrier that runs out is recorded as AWQ_ERR_TIMEOUT in ws. */
awq_status awq_w4a16_moe(const void *X, int64_t T, int64_t hidden, int64_t ldx, const uint8_t *mask,
                         const void *router, int32_t n_experts, int32_t top_k, int32_t renormalize,
                         const int32_t *gu_qweight, const int32_t *gu_qzeros, const void *gu_scales,
                         int64_t inter, const int32_t *dn_qweight, const int32_t *dn_qzeros,
                         const void *dn_scales, const awq_config *cfg, void *Y, int64_t ldy,
                         int32_t *ids, float *weights, void *ws, size_t ws_bytes,
                         awq_stream_t stream);

/* Workspace bytes of awq_w4a16_moe; 0 when the arguments are invalid. */
size_t awq_w4a16_moe_workspace_size(int64_t T, int64_t hidden, int64_t inter, int32_t n_experts,
                                    int32_t top_k, const awq_config *cfg);

/* The end of one block and the start of the next, for T token rows of d:
 *   v' = V rsqrt(mean V^2 + eps) post        (v' = V when post is NULL)
 *   r' = R + c gate v'                       (gate = 1 when gate is NULL)
 *   R_out = RN16(r'),   N_out = RN16( r' rsqrt(mean r'^2 + eps) pre )
 * in fp32 from the inputs to the two roundings; pre (1 when NULL) is the norm
 * weight that awq_fold_inv_scale divides by the next linear's s.
 *   R     device fp16 [T, d], row stride ldr: the residual
 *   V     device fp16 [T, d], row stride ldv: the block's output, or NULL (r' = R;
 *         post and gate must then be NULL)
 *   post, pre   device fp16 [d] or NULL
 *   gate  device fp16 [T, d] with row stride ldg, or [d] with ldg = 0, or NULL
 *   R_out, N_out  device fp16 [T, d], row strides ldro and ldno; either may be
 *         NULL, R_out may be R and N_out may be V (same pointer and stride)
 * Requires d % 8 == 0 and 8 <= d <= 32768, eps >= 0, 1 <= T <= 2^22, row
 * strides multiples of 8 and at least d (but ldg = 0), every pointer 16-byte
 * aligned. */
awq_status awq_block_norm(const void *R, int64_t ldr, const void *V, int64_t ldv, int64_t T,
                          int64_t d, const void *post, const void *gate, int64_t ldg, float c,
                          const void *pre, float eps, void *R_out, int64_t ldro, void *N_out,
                          int64_t ldno, awq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* AWQ_SERVING_H */
