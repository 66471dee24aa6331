/*
 * nvfp4_dit.h -- C ABI of the operators that surround a diffusion transformer
 * block's linear layers: matrix-vector products with 4-bit weights, rotary
 * positions with several axes, and attention to an encoder's states of another
 * length with its backward pass.  Part of libnvfp4.so; every convention of
 * nvfp4.h holds here too (device pointers, the caller's buffers, the current
 * CUDA device, asynchronous calls on `stream`, argument checks on the host
 * before any launch, dev_status).  Non-finite inputs are allowed here and
 * spread as the formulas say, unless a call states otherwise.
 */
#ifndef NVFP4_DIT_H_
#define NVFP4_DIT_H_

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * nvfp4_gemv_w4a16 -- a few rows of activations times 4-bit weights with group
 * scales: the conditioning path of a block (the adaLN modulation has one row
 * per sample), where nvfp4_gemm_w4a16 would compute a whole 256-row tile.
 *   y[m,n] = g * sum_k x[m,k] * e2m1(w[n,k]) * s[n, k / block]  (+ bias[n])
 * Weights and products are exact (in FP16 with a row's values times a power of
 * two where they span few enough binades, in bf16 otherwise), products are added
 * in FP32, g and the bias are applied in FP32, and y is rounded once.
 * x_bf16    [M, K] bf16, row stride ld_x (ld_x >= K, ld_x % 8 == 0; 0: the M rows
 *           are one row in memory, as where samples share their conditioning),
 *           16-byte aligned; 1 <= M <= NVFP4_GEMV_MAX_ROWS (M == 0 is a no-op).
 *           The stride of a single row is checked as any, and not used.
 * w_format  NVFP4_WEIGHTS_NVFP4: w_codes, w_sf, w_scale as nvfp4_quantize
 *           writes a [N, K] tensor (block 16, s = e4m3, g = *w_scale), K % 64 == 0;
 *           NVFP4_WEIGHTS_MX: w_codes, w_sf as nvfp4_mx_quantize writes them
 *           (block 32, s = 2^(byte - 127), g = 1, w_scale ignored), K % 128 == 0.
 *           Either: K <= 2^31 - 128.
 * bias      nullable device FP32 [N].
 * y         [M, N] contiguous in y_dtype (1 <= N < 2^31 - 128).
 * The K range is split over the warps of a CTA and the CTAs of a cluster, whose
 * sums are added in a fixed order: the same call gives the same bits.  (How it is
 * split depends on M, N and K: a row's bits may differ between calls of other M.)
 * One kernel on `stream`, no workspace.
 */
enum { NVFP4_WEIGHTS_NVFP4 = 0, NVFP4_WEIGHTS_MX = 1 };
enum { NVFP4_GEMV_MAX_ROWS = 16 };
nvfp4_status nvfp4_gemv_w4a16(const void *x_bf16, int64_t ld_x, const uint8_t *w_codes, const uint8_t *w_sf,
                              const float *w_scale, int w_format, const float *bias, int64_t M, int64_t N,
                              int64_t K, void *y, int y_dtype, nvfp4_stream_t stream);

/* A [batch, tokens, heads, d] tensor: element (b, l, h, c) at
 * data + b * batch_stride + l * token_stride + h * head_stride + c (strides in
 * elements).  A call reads or writes through it as it says; data and the
 * strides (as bytes) are multiples of 16.  An input may be a broadcast along
 * batch or heads (stride 0); its token stride is at least d.  Every stride of
 * an output is at least d, and no two of its elements share memory.  The
 * stride of an axis of one element is not looked at. */
typedef struct {
    void *data;
    int64_t batch_stride, token_stride, head_stride;
} nvfp4_heads;

/*
 * nvfp4_rotary -- rotary positions with several axes (time, height and width
 * of a video's tokens).  The first R = sum of axis_dims of a head's d values
 * form R/2 pairs; axis a owns axis_dims[a] / 2 of them, in order, and its i-th
 * pair turns by
 *   angle = position[a] * theta^(-2 i / axis_dims[a]),
 *   (u, v) -> (u cos - v sin, u sin + v cos);
 * values past R are copied.  Pair j is (2j, 2j+1) with
 * NVFP4_ROTARY_INTERLEAVED, (j, j + R/2) without.  With NVFP4_ROTARY_INVERSE
 * the angle's sign is flipped: the backward pass (and the inverse) of the call
 * without it.  The angle is formed and reduced to one turn in FP64, cos and sin
 * are FP32 (so far positions lose nothing), the turn is FP32, rounded once.
 * x, out       [B, L, H, d] in dtype (NVFP4_DTYPE_BF16 or NVFP4_DTYPE_F32); out
 *              may be x (same data and strides: in place), not overlap it
 *              otherwise.
 * positions    [B or 1, L, n_axes], contiguous along the axes, element strides
 *              pos_batch_stride (0: shared by the batch) and pos_token_stride;
 *              int32 (NVFP4_POSITION_I32) or FP32 (NVFP4_POSITION_F32).
 * axis_dims    HOST int[n_axes], each even and >= 0, 1 <= n_axes <= 4, sum in
 *              [2, d].
 * theta        > 0 and finite.
 * d % 8 == 0, d <= 256.  One kernel on `stream`.
 */
enum { NVFP4_POSITION_I32 = 0, NVFP4_POSITION_F32 = 1 };
enum { NVFP4_ROTARY_INTERLEAVED = 1, NVFP4_ROTARY_INVERSE = 2 };
nvfp4_status nvfp4_rotary(const nvfp4_heads *x, const void *positions, int pos_dtype, int64_t pos_batch_stride,
                          int64_t pos_token_stride, const int *axis_dims, int n_axes, double theta, int64_t B,
                          int64_t L, int64_t H, int64_t d, int dtype, unsigned flags, const nvfp4_heads *out,
                          nvfp4_stream_t stream);

/*
 * nvfp4_cross_attention -- attention of Lq queries to an encoder's states of
 * another length, each sample with its own number of valid states:
 *   out = softmax(scale * q k^T) v over the keys j < kv_lens[b],
 *   lse = ln sum_j exp(scale * q k_j^T).
 * q, out    [B, Lq, H, d] bf16;  k, v  [B, Lk, Hkv, d] bf16, H % Hkv == 0: query
 *           head h reads key / value head h / (H / Hkv).
 * kv_lens   nullable device int32 [B]: values below 0 count as 0, above Lk as
 *           Lk.  Keys at or past the length are not read into any result,
 *           whatever their memory holds (NaN and infinities too).  A sample
 *           of length 0 gets out = 0 and lse = -infinity.  (A query whose logits
 *           are -infinity at every valid key gets 0 / 0, out = NaN, and
 *           lse = -infinity.)
 * scale     finite and > 0 (usually 1 / sqrt(d)).
 * lse       nullable, out: device FP32 [B, H, Lq] contiguous.
 * d % 8 == 0, 8 <= d <= 128; 0 <= Lq, Lk <= 2^31 - 128; B * H * (Lq + 1) and
 * B * Hkv * (Lk + 1) below 2^31.
 * S = q k^T and P v run on the tensor cores with FP32 accumulation, the softmax
 * is FP32, P is rounded to bf16 for the second product.  One kernel on
 * `stream`.
 */
nvfp4_status nvfp4_cross_attention(const nvfp4_heads *q, const nvfp4_heads *k, const nvfp4_heads *v,
                                   const int32_t *kv_lens, float scale, int64_t B, int64_t H, int64_t Hkv,
                                   int64_t Lq, int64_t Lk, int64_t d, const nvfp4_heads *out, float *lse,
                                   int *dev_status, nvfp4_stream_t stream);

/*
 * nvfp4_cross_attention_backward -- gradients of nvfp4_cross_attention: with
 *   P = exp(scale q k^T - lse), D_i = sum_c grad_out[i,c] out[i,c],
 *   dS = P * (grad_out v^T - D) * scale:
 *   dv = P^T grad_out,  dq = dS k,  dk = dS^T q  (dk, dv summed over the query
 * heads that share a key / value head).  out and lse are the forward call's
 * (for a sample of at most 128 keys D is formed as sum_j P_ij dP_ij, without out).
 * P and dS are rounded to bf16 for the products; sums are FP32.  Keys at or past
 * a sample's length get dk = dv = 0, queries of a sample of length 0 dq = 0.
 * Partial sums are joined in a fixed order: the same call gives the same bits.
 * grad_out, q, out, dq  [B, Lq, H, d];  k, v, dk, dv  [B, Lk, Hkv, d].  Where q,
 *           k or v is a broadcast, its gradient is that of the expanded tensor.
 * workspace device scratch of >= nvfp4_cross_attention_backward_workspace_bytes,
 *           16-byte aligned, not preserved; calls that run at the same time
 *           need workspaces of their own.
 */
size_t nvfp4_cross_attention_backward_workspace_bytes(int64_t B, int64_t H, int64_t Hkv, int64_t Lq, int64_t Lk,
                                                      int64_t d);
nvfp4_status nvfp4_cross_attention_backward(const nvfp4_heads *grad_out, const nvfp4_heads *q, const nvfp4_heads *k,
                                            const nvfp4_heads *v, const nvfp4_heads *out, const float *lse,
                                            const int32_t *kv_lens, float scale, int64_t B, int64_t H, int64_t Hkv,
                                            int64_t Lq, int64_t Lk, int64_t d, const nvfp4_heads *dq,
                                            const nvfp4_heads *dk, const nvfp4_heads *dv, void *workspace,
                                            size_t workspace_bytes, int *dev_status, nvfp4_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_DIT_H_ */
