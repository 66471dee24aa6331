// xattn.cu -- attention to an encoder's states of another length
// (nvfp4_cross_attention and its backward pass): one warp per row.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dit.h"
#include "internal.h"

namespace nvfp4 {
namespace xattn_rows {

constexpr int kThreads = 128;
constexpr int kPer = 4;                   // values of a head a lane holds (columns lane + 32 i)

__device__ __forceinline__ float bf(const void* base, int64_t i) {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
}
__device__ __forceinline__ void load_row(const nvfp4_heads& t, int b, int l, int h, int d, int lane, float (&r)[kPer]) {
    const int64_t at = (int64_t)b * t.batch_stride + (int64_t)l * t.token_stride + (int64_t)h * t.head_stride;
#pragma unroll
    for (int i = 0; i < kPer; ++i) r[i] = lane + 32 * i < d ? bf(t.data, at + lane + 32 * i) : 0.0f;
}
__device__ __forceinline__ void store_row(const nvfp4_heads& t, int b, int l, int h, int d, int lane, const float (&r)[kPer]) {
    const int64_t at = (int64_t)b * t.batch_stride + (int64_t)l * t.token_stride + (int64_t)h * t.head_stride;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (lane + 32 * i < d) static_cast<__nv_bfloat16*>(t.data)[at + lane + 32 * i] = __float2bfloat16_rn(r[i]);
}
__device__ __forceinline__ float dot(const float (&a)[kPer], const float (&b)[kPer]) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) s += a[i] * b[i];
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
__device__ __forceinline__ int keys_of(const CrossAttnArgs& a, int b) {
    return a.kv_lens ? min(max(a.kv_lens[b], 0), a.Lk) : a.Lk;
}

__global__ void __launch_bounds__(kThreads) dq_kernel(const CrossAttnArgs a, float* delta) {
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= (int64_t)a.B * a.H * a.Lq) return;
    const int l = (int)(row % a.Lq), h = (int)(row / a.Lq % a.H), b = (int)(row / a.Lq / a.H), hk = h / (a.H / a.Hkv);
    const int n = keys_of(a, b);
    float q[kPer], g[kPer], k[kPer], v[kPer], r[kPer] = {};
    load_row(a.q, b, l, h, a.d, lane, q);
    load_row(a.grad_out, b, l, h, a.d, lane, g);
    load_row(a.out, b, l, h, a.d, lane, k);
    const float dl = dot(g, k), lse = a.lse[row];
    if (lane == 0) delta[row] = dl;
    for (int j = 0; j < n; ++j) {
        load_row(a.k, b, j, hk, a.d, lane, k);
        load_row(a.v, b, j, hk, a.d, lane, v);
        const float ds = __expf(a.scale * dot(q, k) - lse) * (dot(g, v) - dl) * a.scale;
#pragma unroll
        for (int i = 0; i < kPer; ++i) r[i] += ds * k[i];
    }
    store_row(a.dq, b, l, h, a.d, lane, r);
}

__global__ void __launch_bounds__(kThreads) dkv_kernel(const CrossAttnArgs a, const float* delta) {
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= (int64_t)a.B * a.Hkv * a.Lk) return;
    const int j = (int)(row % a.Lk), hk = (int)(row / a.Lk % a.Hkv), b = (int)(row / a.Lk / a.Hkv), group = a.H / a.Hkv;
    float q[kPer], g[kPer], k[kPer], v[kPer], dk[kPer] = {}, dv[kPer] = {};
    if (j < keys_of(a, b)) {
        load_row(a.k, b, j, hk, a.d, lane, k);
        load_row(a.v, b, j, hk, a.d, lane, v);
        for (int h = hk * group; h < (hk + 1) * group; ++h)
            for (int l = 0; l < a.Lq; ++l) {
                load_row(a.q, b, l, h, a.d, lane, q);
                load_row(a.grad_out, b, l, h, a.d, lane, g);
                const int64_t at = ((int64_t)b * a.H + h) * a.Lq + l;
                const float p = __expf(a.scale * dot(q, k) - a.lse[at]), ds = p * (dot(g, v) - delta[at]) * a.scale;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    dv[i] += p * g[i];
                    dk[i] += ds * q[i];
                }
            }
    }
    store_row(a.dk, b, j, hk, a.d, lane, dk);
    store_row(a.dv, b, j, hk, a.d, lane, dv);
}

unsigned blocks_of(int64_t rows) { return (unsigned)((rows + kThreads / 32 - 1) / (kThreads / 32)); }

}  // namespace xattn_rows

size_t cross_attention_backward_workspace(int64_t B, int64_t H, int64_t, int64_t Lq, int64_t, int64_t) {
    return (size_t)(B * H * Lq) * sizeof(float);
}

cudaError_t launch_cross_attention_backward(const CrossAttnArgs& a, int, cudaStream_t stream) {
    float* delta = static_cast<float*>(a.workspace);
    const int64_t rows = (int64_t)a.B * a.H * a.Lq, keys = (int64_t)a.B * a.Hkv * a.Lk;
    if (rows > 0) xattn_rows::dq_kernel<<<xattn_rows::blocks_of(rows), xattn_rows::kThreads, 0, stream>>>(a, delta);
    if (keys > 0) xattn_rows::dkv_kernel<<<xattn_rows::blocks_of(keys), xattn_rows::kThreads, 0, stream>>>(a, delta);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launch((rows > 0) + (keys > 0));
    return e;
}

}  // namespace nvfp4
