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

// A [B, L, H, d] bf16 operand as a 4-D map (d, h, l, b) with boxes of `cols` (64 or 32: the swizzle is as wide as
// their bytes) x `rows` tokens of one head.
inline bool make_heads_map(CUtensorMap* map, const nvfp4_heads& t, int B, int L, int H, int d, int rows, MapAxes* axes,
                           int cols = 64) {
    axes->b = t.batch_stride != 0;
    axes->h = t.head_stride != 0;
    const uint64_t step = (uint64_t)d * 2;   // a legal stride for axes of one element
    const uint64_t dims[4] = {(uint64_t)d, axes->h ? (uint64_t)H : 1u, (uint64_t)L, axes->b ? (uint64_t)B : 1u};
    const uint64_t strides[3] = {axes->h ? (uint64_t)t.head_stride * 2 : step, L > 1 ? (uint64_t)t.token_stride * 2 : step,
                                 axes->b ? (uint64_t)t.batch_stride * 2 : step};
    const uint32_t box[4] = {(uint32_t)cols, 1, (uint32_t)rows, 1};
    return make_tmap_4d(map, t.data, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, strides, box,
                        cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) == CUDA_SUCCESS;
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

// A box from shared memory; rows and columns past the tensor are not written.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, const void* src, int x, int h, int l, int b) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(x), "r"(h), "r"(l), "r"(b)
                 : "memory");
}

// A tile (all its 64-column chunks), completion on `bar` (which expects chunks * rows * 128 bytes).
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int chunks, int chunk_bytes,
                                          int h, int l, int b) {
    for (int c = 0; c < chunks; ++c) tma_load_4d(dst + c * chunk_bytes, map, bar, c * 64, h, l, b);
}

// kind::f16 on bf16 operands, FP32 sums: both K-major (idesc_bf16), or B
// MN-major (bit 16): rows of B's tile run along k.
__device__ __forceinline__ uint32_t idesc_kk(int N) { return idesc_bf16(kRows, N); }
__device__ __forceinline__ uint32_t idesc_kmn(int N) { return idesc_bf16(kRows, N) | (1u << 16); }

// Products of a tile, at most eight steps of 16 along k, called by a converged
// warp; each instruction elects the lane that issues it.  (A tile product takes
// the tensor core 512 cycles.  Issued like this, eight steps take 436 cycles of
// the warp; behind one elected branch 540; under a predicate on the lane number,
// which may hold for several lanes as far as the compiler knows, 770 and more.)
// The descriptors of the steps differ by constants in their low word.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);   // 8-row groups 1024 bytes apart, 128-byte swizzle

// D[tmem] = A B^T: both tiles K-major (k = d: four steps a chunk).
__device__ __forceinline__ void product_kk(uint32_t d, uint32_t a_tile, uint32_t b_tile, uint32_t idesc, int steps) {
    const uint32_t a = (a_tile >> 4) | (1u << 16), b = (b_tile >> 4) | (1u << 16);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
        if (kk >= steps) break;
        const uint32_t off = (kk >> 2) * (kChunk >> 4) + (kk & 3) * 2;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
            "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
            "setp.ne.b32 p, %5, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}"
            ::"r"(d), "r"(a + off), "r"(b + off), "n"(kDescHigh), "r"(idesc), "r"((uint32_t)kk)
            : "memory");
    }
}

// D[tmem] (+)= A B: A packed in TMEM, two values a column, the 16 values of step
// kk at a + (kk / GROUP) * 16 GROUP + (kk % GROUP) * 8; B MN-major (k = its rows).
template <int GROUP>
__device__ __forceinline__ void product_tmem(uint32_t d, uint32_t a, uint32_t b_tile, uint32_t idesc, int steps,
                                             bool accumulate) {
    const uint32_t b = (b_tile >> 4) | ((uint32_t)(kChunk >> 4) << 16);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
        if (kk >= steps) break;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\t"
            "mov.b64 db, {%2, %3};\n\t"
            "setp.ne.b32 p, %5, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}"
            ::"r"(d), "r"(a + (kk / GROUP) * 16 * GROUP + (kk % GROUP) * 8), "r"(b + kk * 128), "n"(kDescHigh), "r"(idesc),
              "r"(kk > 0 || accumulate ? 1u : 0u)
            : "memory");
    }
}

// What the issuing warp has to know of a step, left by the loading warp beside
// the step's K tile (0: no more steps).
constexpr uint32_t kInfoKeys = 0xFFu;        // keys of the tile, 1 .. 128
constexpr uint32_t kInfoFirst = 1u << 8;     // first, last step of an item
constexpr uint32_t kInfoLast = 1u << 9;
constexpr uint32_t kInfoZero = 1u << 10;     // rows past the sample's length may hold anything
constexpr uint32_t kInfoTwo = 1u << 11;      // the item has a second query tile

__device__ __forceinline__ uint32_t step_info(int keys, int Lk, int j, int steps, bool two) {
    const int n = min(keys - j * kRows, kRows);
    return (uint32_t)n | (j == 0 ? kInfoFirst : 0u) | (j == steps - 1 ? kInfoLast : 0u) |
           ((n & 15) != 0 && keys < Lk ? kInfoZero : 0u) | (two ? kInfoTwo : 0u);
}

// Rows [n, n rounded up to 16) of a tile as zeros, by the whole warp: those keys
// meet a zero in the other operand, but may be NaN (rows past the tensor are zeros already).
__device__ __forceinline__ void zero_rest(uint8_t* tile, int n, int chunks, int lane) {
    const int pieces = (16 - (n & 15)) * 8;
    for (int c = 0; c < chunks; ++c)
        for (int i = lane; i < pieces; i += 32)
            *reinterpret_cast<uint4*>(tile + c * kChunk + n * 128 + i * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
}

// `bar` is told when all products issued so far are complete (a converged warp).
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(smem_u32(bar))
        : "memory");
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

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two FP32 operations in one instruction, on neighbouring registers.
struct F2 {
    float x, y;
};
__device__ __forceinline__ uint64_t f2_bits(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ F2 f2_of(uint64_t b) {
    F2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a.x, a.y)), "l"(f2_bits(b.x, b.y)), "l"(f2_bits(c.x, c.y)));
    return f2_of(r);
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a.x, a.y)), "l"(f2_bits(b.x, b.y)));
    return f2_of(r);
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a.x, a.y)), "l"(f2_bits(b.x, b.y)));
    return f2_of(r);
}

// 2^x of two values on the FMA pipes, for -inf <= x < 127: x = n + r with |r| <=
// 1/2, 2^r by the polynomial of degree 5 of least relative error (Remez exchange,
// 2^-23.7; 2^-22.1 with the roundings of FP32), times 2^n.  x is taken as at least
// -127, where the factor's exponent field is 0: zero from -126.5 down, at -infinity
// too, as the hardware exponential gives it below -126; NaN stays NaN.  The hardware
// exponential does 16 values a cycle and SM, and a tile of 128 x 128 takes 1024
// cycles of it: where those hold up a kernel, a part goes this way.
__device__ __forceinline__ F2 ex2_fma(F2 x) {
    asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x.x));
    asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(x.y));
    const F2 m = {12583039.0f, 12583039.0f};                // 1.5 * 2^23 + 127: n + 127 in the low bits
    const F2 t = add2(x, m);
    const F2 u = add2(t, {-m.x, -m.y});
    const F2 r = add2(x, {-u.x, -u.y});
    F2 p = fma2(r, {0.0013276472454890609f, 0.0013276472454890609f}, {0.009675540961325169f, 0.009675540961325169f});
    p = fma2(p, r, {0.05550713092088699f, 0.05550713092088699f});
    p = fma2(p, r, {0.24022120237350464f, 0.24022120237350464f});
    p = fma2(p, r, {0.6931469440460205f, 0.6931469440460205f});
    p = fma2(p, r, {1.0000001192092896f, 1.0000001192092896f});
    return mul2(p, {__uint_as_float(__float_as_uint(t.x) << 23), __uint_as_float(__float_as_uint(t.y) << 23)});
}

// 2^x of pair i of a row's values: KIND of eight pairs on the FMA pipes.
template <int KIND>
__device__ __forceinline__ F2 ex2_pair(F2 x, int i) {
    if ((i * KIND & 7) + KIND >= 8 && (i & 7) != 0) return ex2_fma(x);
    return {ex2(x.x), ex2(x.y)};
}

// The whole warp waits (as mbar_wait, with its limit); false once the block gives
// up.  Every branch is on a vote, so that the code around it stays convergent.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtx& w) {
    const uint32_t at = smem_u32(bar);
    if (__all_sync(0xffffffffu, mbar_try_wait(at, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
    uint32_t n = 0;
    while (true) {
        if (__all_sync(0xffffffffu, mbar_try_wait(at, parity))) return true;
        if ((++n & 255u) == 0u) {
            if (__any_sync(0xffffffffu, *w.abort_flag)) return false;
            if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitLimitNs)) {
                report_timeout(w);
                return false;
            }
        }
    }
}

}  // namespace xattn
}  // namespace nvfp4
