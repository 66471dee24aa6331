// dit.h -- launch-side declarations of the kernels behind nvfp4_dit.h (not
// part of the public C ABI).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/nvfp4_dit.h"

namespace nvfp4 {

struct GemvArgs {
    const uint16_t* x;
    int64_t ld_x;
    const uint8_t* w_codes;
    const uint8_t* w_sf;
    const float* w_scale;     // null: 1 (MX weights)
    bool mx;
    const float* bias;        // nullable
    int M, N, K;
    void* y;
    bool y_f32;
};

cudaError_t launch_gemv(const GemvArgs& a, int num_sms, cudaStream_t stream);

constexpr int kRotaryMaxPairs = 128;
constexpr int kRotaryMaxAxes = 4;

struct RotaryArgs {
    nvfp4_heads x, out;
    const void* positions;
    int64_t pos_batch_stride, pos_token_stride;
    bool pos_f32;
    int n_axes, pairs;
    int axis_pairs[kRotaryMaxAxes];
    double theta;
    int64_t B, L, H, d;
    bool f32, interleaved, inverse;
};

cudaError_t launch_rotary(const RotaryArgs& a, int num_sms, cudaStream_t stream);

struct CrossAttnArgs {
    nvfp4_heads q, k, v, out;
    const int32_t* kv_lens;   // nullable
    float scale;
    int B, H, Hkv, Lq, Lk, d;
    float* lse;               // [B, H, Lq]; nullable in the forward call
    int* dev_status;
    // backward only
    nvfp4_heads grad_out, dq, dk, dv;
    void* workspace;
};

namespace xattn {
cudaError_t launch_forward_few(const CrossAttnArgs& a, int num_sms, cudaStream_t stream);      // at most 16 rows a key / value head
}
cudaError_t launch_cross_attention(const CrossAttnArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_cross_attention_backward(const CrossAttnArgs& a, int num_sms, cudaStream_t stream);
size_t cross_attention_backward_workspace(int64_t B, int64_t H, int64_t Hkv, int64_t Lq, int64_t Lk, int64_t d);

}  // namespace nvfp4
