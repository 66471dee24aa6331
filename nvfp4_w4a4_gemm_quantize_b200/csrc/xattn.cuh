// xattn.cuh -- what the cross-attention kernels (forward and backward) share:
// operand descriptions, tensor-core and TMEM wrappers, tile geometry.
//
// Tiles are 128 rows of a head's d values (tokens of one sample and head), kept
// as ceil(d / 64) chunks of 128 rows x 128 bytes in the 128-byte swizzle; TMA
// fills columns past d and rows past the tensor with zeros, so d is any
// multiple of 8 up to 128 at run time: a product over d takes ceil(d / 16)
// steps, a product into d has N = d rounded up to 16.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dit.h"
#include "internal.h"
#include "ptx.cuh"
#include "tmap.h"

namespace nvfp4 {
namespace xattn {

constexpr int kRows = 128;                   // rows of a tile
constexpr int kChunk = kRows * 128;          // 16 KB: 64 columns of a tile
constexpr int kSmemLimit = 232448;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Whether a tensor map has a batch and a head axis (0: broadcast or one element).
struct MapAxes {
    int b, h;
};

// A [B, L, H, d] bf16 operand as a 4-D map (d, h, l, b) with boxes of 64 columns x `rows` tokens of one head.
inline bool make_heads_map(CUtensorMap* map, const nvfp4_heads& t, int B, int L, int H, int d, int rows, MapAxes* axes) {
    axes->b = t.batch_stride != 0;
    axes->h = t.head_stride != 0;
    const uint64_t step = (uint64_t)d * 2;   // a legal stride for axes of one element
    const uint64_t dims[4] = {(uint64_t)d, axes->h ? (uint64_t)H : 1u, (uint64_t)L, axes->b ? (uint64_t)B : 1u};
    const uint64_t strides[3] = {axes->h ? (uint64_t)t.head_stride * 2 : step, L > 1 ? (uint64_t)t.token_stride * 2 : step,
                                 axes->b ? (uint64_t)t.batch_stride * 2 : step};
    const uint32_t box[4] = {64, 1, (uint32_t)rows, 1};
    return make_tmap_4d(map, t.data, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ==
           CUDA_SUCCESS;
}

// Valid keys of sample b.
__device__ __forceinline__ int keys_of(const int32_t* kv_lens, int b, int Lk) {
    return kv_lens ? min(max(__ldg(kv_lens + b), 0), Lk) : Lk;
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int h, int l, int b) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(h), "r"(l), "r"(b)
        : "memory");
}

// A tile (all its 64-column chunks), completion on `bar` (which expects chunks * rows * 128 bytes).
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int chunks, int chunk_bytes,
                                          int h, int l, int b) {
    for (int c = 0; c < chunks; ++c) tma_load_4d(dst + c * chunk_bytes, map, bar, c * 64, h, l, b);
}

// D[tmem] (+)= A[tmem] * B[smem], bf16, A packed two values a column.
__device__ __forceinline__ void tc_mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// kind::f16 on bf16 operands, FP32 sums: both K-major (idesc_bf16), or B
// MN-major (bit 16): rows of B's tile run along k.
__device__ __forceinline__ uint32_t idesc_kk(int N) { return idesc_bf16(kRows, N); }
__device__ __forceinline__ uint32_t idesc_kmn(int N) { return idesc_bf16(kRows, N) | (1u << 16); }

// A tile as a K-major operand (k = d), step kk: 16 columns on; chunks of `chunk_bytes`.
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t tile, int kk, int chunk_bytes) {
    return sdesc_kmajor_sw128(tile + (kk >> 2) * chunk_bytes + (kk & 3) * 32);
}
// A tile as an MN-major B operand (k = its rows, n = d), step kk: 16 rows on.
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t tile, int kk, int chunk_bytes) {
    return make_sdesc(tile + kk * 2048, chunk_bytes, 1024, 2);
}

__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The whole warp waits; false once the block gives up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtx& w) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, w) ? 1 : 0) != 0;
}

}  // namespace xattn
}  // namespace nvfp4
