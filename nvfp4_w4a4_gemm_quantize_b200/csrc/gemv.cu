// gemv.cu -- a few rows of activations times 4-bit weights with group scales
// (nvfp4_gemv_w4a16): one warp per output feature, FP32 sums.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dit.h"
#include "internal.h"
#include "ptx.cuh"

namespace nvfp4 {
namespace gemv {

constexpr int kThreads = 128;

__device__ __forceinline__ float e2m1(uint32_t c) {
    const uint32_t e = (c >> 1) & 3u, m = c & 1u;
    const float v = e == 0 ? 0.5f * (float)m : __uint_as_float((126u + e) << 23) * (1.0f + 0.5f * (float)m);
    return (c & 8u) ? -v : v;
}

__global__ void __launch_bounds__(kThreads) gemv_kernel(const GemvArgs a) {
    const int lane = threadIdx.x & 31, n = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (n >= a.N) return;
    const int block = a.mx ? 32 : 16, kb = a.K / block;
    for (int m = 0; m < a.M; ++m) {
        float acc = 0.0f;
        for (int k = 2 * lane; k < a.K; k += 64) {
            const uint32_t byte = a.w_codes[(int64_t)n * (a.K / 2) + k / 2];
            const int c = k / block;
            const uint32_t sf = a.w_sf[((int64_t)(n / 128) * (kb / 4) + c / 4) * 512 + (n % 32) * 16 + ((n % 128) / 32) * 4 + c % 4];
            const float s = a.mx ? ldexpf(1.0f, (int)sf - 127) : e4m3_to_f32(sf);
            const uint16_t* x = a.x + (int64_t)m * a.ld_x + k;
            acc += __uint_as_float((uint32_t)x[0] << 16) * (e2m1(byte & 15u) * s) +
                   __uint_as_float((uint32_t)x[1] << 16) * (e2m1(byte >> 4) * s);
        }
        for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if (lane == 0) {
            float y = (a.w_scale ? *a.w_scale : 1.0f) * acc;
            if (a.bias) y += a.bias[n];
            if (a.y_f32) static_cast<float*>(a.y)[(int64_t)m * a.N + n] = y;
            else static_cast<__nv_bfloat16*>(a.y)[(int64_t)m * a.N + n] = __float2bfloat16_rn(y);
        }
    }
}

}  // namespace gemv

cudaError_t launch_gemv(const GemvArgs& a, int, cudaStream_t stream) {
    gemv::gemv_kernel<<<(a.N + 3) / 4, gemv::kThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(1);
    return e;
}

}  // namespace nvfp4
