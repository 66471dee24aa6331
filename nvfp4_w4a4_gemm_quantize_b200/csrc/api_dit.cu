// api_dit.cu -- the C ABI of include/nvfp4_dit.h: host-side argument checks and
// the kernel launches.  No call allocates device memory and none synchronizes
// the host.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "dit.h"
#include "internal.h"

using namespace nvfp4;

namespace {

constexpr int64_t kMaxInt = (int64_t)1 << 31;
constexpr int64_t kMaxTiled = kMaxInt - 128;           // lengths that kernels round up to tiles of 128 in 32 bits
constexpr int64_t kMaxStride = (int64_t)1 << 37;       // elements: below the 2^40 bytes of a tensor map's stride

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
nvfp4_status cuda_status(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

// A [B, L, H, d] operand: present, strides in range, 16-byte steps of
// elements of `size` bytes.  `written`: no two elements may share memory.
nvfp4_status check_heads(const nvfp4_heads* t, int64_t B, int64_t L, int64_t H, int64_t d, int size, bool written) {
    if (!t || !t->data) return NVFP4_ERR_INVALID_ARG;
    const int64_t strides[3] = {t->batch_stride, t->token_stride, t->head_stride}, dims[3] = {B, L, H};
    for (int i = 0; i < 3; ++i) {
        if (dims[i] <= 1) continue;                    // never multiplied by more than 0
        if (strides[i] < 0 || strides[i] >= kMaxStride) return NVFP4_ERR_INVALID_ARG;
        if (written && strides[i] < d) return NVFP4_ERR_INVALID_ARG;
        if ((strides[i] * size) % 16 != 0) return NVFP4_ERR_MISALIGNED;
    }
    // only a batch or head axis may be a broadcast
    if (L > 1 && t->token_stride < d) return NVFP4_ERR_INVALID_ARG;
    return aligned16(t->data) ? NVFP4_OK : NVFP4_ERR_MISALIGNED;
}

// The strides of axes of one element set to 0, so that kernels may multiply by them.
nvfp4_heads tidy(const nvfp4_heads* t, int64_t B, int64_t L, int64_t H) {
    nvfp4_heads r = *t;
    if (B <= 1) r.batch_stride = 0;
    if (L <= 1) r.token_stride = 0;
    if (H <= 1) r.head_stride = 0;
    return r;
}

nvfp4_status check_attention_sizes(int64_t B, int64_t H, int64_t Hkv, int64_t Lq, int64_t Lk, int64_t d, float scale,
                                   const int32_t* kv_lens) {
    if (B < 0 || H <= 0 || Hkv <= 0 || Lq < 0 || Lk < 0 || d <= 0) return NVFP4_ERR_INVALID_ARG;
    if (!(scale > 0.0f) || std::isinf(scale)) return NVFP4_ERR_INVALID_ARG;
    if (H % Hkv != 0) return NVFP4_ERR_INVALID_ARG;
    if (d % 8 != 0 || d > 128) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (B >= kMaxInt || H >= kMaxInt || Lq > kMaxTiled || Lk > kMaxTiled || B * H >= kMaxInt ||
        B * H * (Lq + 1) >= kMaxInt || B * Hkv * (Lk + 1) >= kMaxInt)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned4(kv_lens)) return NVFP4_ERR_MISALIGNED;
    return NVFP4_OK;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_gemv_w4a16(const void* x_bf16, int64_t ld_x, const uint8_t* w_codes, const uint8_t* w_sf,
                              const float* w_scale, int w_format, const float* bias, int64_t M, int64_t N, int64_t K,
                              void* y, int y_dtype, nvfp4_stream_t stream) {
    if (M < 0 || N <= 0 || K <= 0 || (ld_x < K && ld_x != 0)) return NVFP4_ERR_INVALID_ARG;
    if (w_format != NVFP4_WEIGHTS_NVFP4 && w_format != NVFP4_WEIGHTS_MX) return NVFP4_ERR_INVALID_ARG;
    if (y_dtype != NVFP4_DTYPE_BF16 && y_dtype != NVFP4_DTYPE_F32) return NVFP4_ERR_INVALID_ARG;
    const bool mx = w_format == NVFP4_WEIGHTS_MX;
    if (M > NVFP4_GEMV_MAX_ROWS || K % (mx ? 128 : 64) != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (N >= kMaxTiled || K > kMaxTiled || ld_x >= kMaxStride) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return NVFP4_OK;                 /* nothing to read or write */
    if (!x_bf16 || !w_codes || !w_sf || (!mx && !w_scale) || !y) return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(x_bf16) || !aligned16(w_codes) || !aligned16(w_sf) || !aligned16(y) || (M > 1 && ld_x % 8 != 0) ||
        !aligned4(w_scale) || !aligned4(bias))
        return NVFP4_ERR_MISALIGNED;
    int sms = 0;
    const nvfp4_status st = device_ok(&sms);
    if (st != NVFP4_OK) return st;
    GemvArgs a{static_cast<const uint16_t*>(x_bf16), M > 1 ? ld_x : K, w_codes, w_sf, mx ? nullptr : w_scale, mx,
               bias, (int)M, (int)N, (int)K, y, y_dtype == NVFP4_DTYPE_F32};
    return cuda_status(launch_gemv(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_rotary(const nvfp4_heads* x, const void* positions, int pos_dtype, int64_t pos_batch_stride,
                          int64_t pos_token_stride, const int* axis_dims, int n_axes, double theta, int64_t B,
                          int64_t L, int64_t H, int64_t d, int dtype, unsigned flags, const nvfp4_heads* out,
                          nvfp4_stream_t stream) {
    if (B < 0 || L < 0 || H < 0 || d <= 0 || !axis_dims || n_axes < 1 || n_axes > kRotaryMaxAxes)
        return NVFP4_ERR_INVALID_ARG;
    if (dtype != NVFP4_DTYPE_BF16 && dtype != NVFP4_DTYPE_F32) return NVFP4_ERR_INVALID_ARG;
    if (pos_dtype != NVFP4_POSITION_I32 && pos_dtype != NVFP4_POSITION_F32) return NVFP4_ERR_INVALID_ARG;
    if ((flags & ~(unsigned)(NVFP4_ROTARY_INTERLEAVED | NVFP4_ROTARY_INVERSE)) != 0u) return NVFP4_ERR_INVALID_ARG;
    if (!(theta > 0.0) || std::isinf(theta)) return NVFP4_ERR_INVALID_ARG;
    if (d % 8 != 0 || d > 2 * kRotaryMaxPairs) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    RotaryArgs a{};
    int64_t sum = 0;
    for (int i = 0; i < n_axes; ++i) {
        if (axis_dims[i] < 0 || axis_dims[i] % 2 != 0) return NVFP4_ERR_INVALID_ARG;
        a.axis_pairs[i] = axis_dims[i] / 2;
        sum += axis_dims[i];
    }
    if (sum < 2 || sum > d) return NVFP4_ERR_INVALID_ARG;
    if (B >= kMaxInt || L >= kMaxInt || B * L >= kMaxInt || H > ((int64_t)1 << 26) / d)
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (pos_batch_stride < 0 || pos_token_stride < 0 || pos_batch_stride >= kMaxStride ||
        pos_token_stride >= kMaxStride)
        return NVFP4_ERR_INVALID_ARG;
    if (B == 0 || L == 0 || H == 0) return NVFP4_OK;
    if (!positions) return NVFP4_ERR_INVALID_ARG;
    const int size = dtype == NVFP4_DTYPE_F32 ? 4 : 2;
    nvfp4_status st = check_heads(x, B, L, H, d, size, false);
    if (st != NVFP4_OK) return st;
    st = check_heads(out, B, L, H, d, size, true);
    if (st != NVFP4_OK) return st;
    if (!aligned4(positions)) return NVFP4_ERR_MISALIGNED;
    int sms = 0;
    st = device_ok(&sms);
    if (st != NVFP4_OK) return st;
    a.x = tidy(x, B, L, H);
    a.out = tidy(out, B, L, H);
    a.positions = positions;
    a.pos_batch_stride = pos_batch_stride;
    a.pos_token_stride = pos_token_stride;
    a.pos_f32 = pos_dtype == NVFP4_POSITION_F32;
    a.n_axes = n_axes;
    a.pairs = (int)(sum / 2);
    a.theta = theta;
    a.B = B;
    a.L = L;
    a.H = H;
    a.d = d;
    a.f32 = dtype == NVFP4_DTYPE_F32;
    a.interleaved = (flags & NVFP4_ROTARY_INTERLEAVED) != 0u;
    a.inverse = (flags & NVFP4_ROTARY_INVERSE) != 0u;
    return cuda_status(launch_rotary(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_cross_attention(const nvfp4_heads* q, const nvfp4_heads* k, const nvfp4_heads* v,
                                   const int32_t* kv_lens, float scale, int64_t B, int64_t H, int64_t Hkv, int64_t Lq,
                                   int64_t Lk, int64_t d, const nvfp4_heads* out, float* lse, int* dev_status,
                                   nvfp4_stream_t stream) {
    nvfp4_status st = check_attention_sizes(B, H, Hkv, Lq, Lk, d, scale, kv_lens);
    if (st != NVFP4_OK) return st;
    if (B == 0 || Lq == 0) return NVFP4_OK;
    if ((st = check_heads(q, B, Lq, H, d, 2, false)) != NVFP4_OK) return st;
    if ((st = check_heads(out, B, Lq, H, d, 2, true)) != NVFP4_OK) return st;
    if (Lk > 0) {
        if ((st = check_heads(k, B, Lk, Hkv, d, 2, false)) != NVFP4_OK) return st;
        if ((st = check_heads(v, B, Lk, Hkv, d, 2, false)) != NVFP4_OK) return st;
    }
    if (!aligned4(lse)) return NVFP4_ERR_MISALIGNED;
    int sms = 0;
    if ((st = device_ok(&sms)) != NVFP4_OK) return st;
    CrossAttnArgs a{};
    a.q = tidy(q, B, Lq, H);
    a.out = tidy(out, B, Lq, H);
    if (Lk > 0) {
        a.k = tidy(k, B, Lk, Hkv);
        a.v = tidy(v, B, Lk, Hkv);
    }
    a.kv_lens = kv_lens;
    a.scale = scale;
    a.B = (int)B;
    a.H = (int)H;
    a.Hkv = (int)Hkv;
    a.Lq = (int)Lq;
    a.Lk = (int)Lk;
    a.d = (int)d;
    a.lse = lse;
    a.dev_status = dev_status;
    return cuda_status(launch_cross_attention(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t nvfp4_cross_attention_backward_workspace_bytes(int64_t B, int64_t H, int64_t Hkv, int64_t Lq, int64_t Lk,
                                                      int64_t d) {
    if (check_attention_sizes(B, H, Hkv, Lq, Lk, d, 1.0f, nullptr) != NVFP4_OK) return 0;
    return cross_attention_backward_workspace(B, H, Hkv, Lq, Lk, d);
}

nvfp4_status nvfp4_cross_attention_backward(const nvfp4_heads* grad_out, const nvfp4_heads* q, const nvfp4_heads* k,
                                            const nvfp4_heads* v, const nvfp4_heads* out, const float* lse,
                                            const int32_t* kv_lens, float scale, int64_t B, int64_t H, int64_t Hkv,
                                            int64_t Lq, int64_t Lk, int64_t d, const nvfp4_heads* dq,
                                            const nvfp4_heads* dk, const nvfp4_heads* dv, void* workspace,
                                            size_t workspace_bytes, int* dev_status, nvfp4_stream_t stream) {
    nvfp4_status st = check_attention_sizes(B, H, Hkv, Lq, Lk, d, scale, kv_lens);
    if (st != NVFP4_OK) return st;
    if (B == 0 || (Lq == 0 && Lk == 0)) return NVFP4_OK;
    if (Lq > 0) {
        const nvfp4_heads* rows[4] = {grad_out, q, out, dq};
        for (int i = 0; i < 4; ++i)
            if ((st = check_heads(rows[i], B, Lq, H, d, 2, i == 3)) != NVFP4_OK) return st;
        if (!lse) return NVFP4_ERR_INVALID_ARG;
    }
    if (Lk > 0) {
        const nvfp4_heads* cols[4] = {k, v, dk, dv};
        for (int i = 0; i < 4; ++i)
            if ((st = check_heads(cols[i], B, Lk, Hkv, d, 2, i >= 2)) != NVFP4_OK) return st;
    }
    const size_t need = cross_attention_backward_workspace(B, H, Hkv, Lq, Lk, d);
    if (need > 0 && (!workspace || workspace_bytes < need)) return NVFP4_ERR_WORKSPACE;
    if (!aligned16(workspace) || !aligned4(lse)) return NVFP4_ERR_MISALIGNED;
    int sms = 0;
    if ((st = device_ok(&sms)) != NVFP4_OK) return st;
    CrossAttnArgs a{};
    if (Lq > 0) {
        a.grad_out = tidy(grad_out, B, Lq, H);
        a.q = tidy(q, B, Lq, H);
        a.out = tidy(out, B, Lq, H);
        a.dq = tidy(dq, B, Lq, H);
    }
    if (Lk > 0) {
        a.k = tidy(k, B, Lk, Hkv);
        a.v = tidy(v, B, Lk, Hkv);
        a.dk = tidy(dk, B, Lk, Hkv);
        a.dv = tidy(dv, B, Lk, Hkv);
    }
    a.kv_lens = kv_lens;
    a.scale = scale;
    a.B = (int)B;
    a.H = (int)H;
    a.Hkv = (int)Hkv;
    a.Lq = (int)Lq;
    a.Lk = (int)Lk;
    a.d = (int)d;
    a.lse = const_cast<float*>(lse);
    a.dev_status = dev_status;
    a.workspace = workspace;
    return cuda_status(launch_cross_attention_backward(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
