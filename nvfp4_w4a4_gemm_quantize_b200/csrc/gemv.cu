// gemv.cu -- a few rows of activations times 4-bit weights with group scales
// (nvfp4_gemv_w4a16):
//   y[m,n] = g sum_k x[m,k] e2m1(w[n,k]) s[n, k / block] (+ bias[n]),  M <= 16.
// Bound by reading the weights once, N K / 2 + N K / block bytes, and close behind
// by the instructions that decode them.
//
// The weights are the A operand of m16n8k16 products (16 output features, 8 rows
// of x), so one decoded register serves every row of x.  An item is 32 features x
// 128 k: features 128 b + 8 q + (0 .. 7) + 32 (0 .. 3), whose scales of 64 k are
// one 16-byte word of the scale layout for each lane.  A lane reads 16 code bytes
// a feature, 32 neighbouring k: the order of k within a product is free as long as
// x comes in the same one, so nothing is shuffled.
// Work: a cluster of 1 to 8 blocks of 16 warps takes a range of the 32-feature
// units; its blocks split k (each keeps its part of x in shared memory), a block's
// warps split the block's items evenly, in order.  Sums are joined in a fixed order
// (warps, then blocks over distributed shared memory): results do not depend on
// timing and need no workspace.
//
// Decoding: the products run in FP16 where that is exact, which halves the decoding
// instructions (the hardware has E2M1 pairs to FP16 pairs; to bf16 it takes shifts
// and masks).  Rows of x are kept times a power of two that puts their largest
// value (of the block's k range) at 2^14; 8 significant bits are exact in FP16 down
// to 2^-17, so a range whose values span at most 31 binades is exact.  E2M1 times
// E4M3 is exact (6 bits, 2^-10 .. 2688); for a single row, and for E8M0 scales, the
// products are of unscaled codes, arranged so that their sums come apart by block,
// and the scales multiply those in FP32.  A block that finds a wider range, or a
// value that is not finite, decodes to bf16 instead.
// B200: 5120 -> 20480, NVFP4, one row 19.7 us (59 MB: 9.0 at the copy rate): the ALU
// pipe is 47 % busy, the issue slots 45 %, DRAM 44 %, so nothing bounds it but its
// start (x and the first items, 5 us, in which nothing is decoded) and the latency of
// a warp's one item at a time.  20480 -> 5120, MX, sixteen rows 36.9 us (15 clusters
// of 8 hold 120 of the 148 SMs; x 10, the join 5, issue slots 50 % busy).
// Items through shared memory, four ahead, against two in registers: 21 and 36 us
// against 24 and 40.5; 2 x 4 blocks and a 128-feature tile each: 28 and 48.
#include <atomic>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dit.h"
#include "internal.h"
#include "ptx.cuh"

namespace nvfp4 {
namespace gemv {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kStepK = 128;                   // k of an item
constexpr int kUnitN = 32;                    // features of an item
constexpr int kMaxCluster = 8;
constexpr int kSmemLimit = 232448 - 2048;     // dynamic

struct Params {
    GemvArgs a;
    int units;                                // 32-feature units
    int steps;                                // ceil(K / 128)
    int segment;                              // steps of x kept at a time
    int unit_chunk;                           // units whose sums are kept at a time
    int kb4;                                  // scale atoms along k: K / (4 block)
    int units_each, units_more, steps_each, steps_more;     // of a cluster, of a block: the first `more` have one more
};

// An item of a lane: 16 code bytes and the scales of its four features.
struct Item {
    uint4 codes[4];
    uint4 sf;                                 // word i: four blocks of feature i
};
constexpr int kItemBytes = 5 * 512;           // of a warp

// Items a warp has in shared memory, the current one and those on their way (asynchronous copies: with the next two in
// registers there was room for 12 warps, and x waited for the weights behind it): as many as leave x its room.
template <int NT>
constexpr int kDepth = NT == 1 ? 4 : 2;
template <int NT>
constexpr int kXBytes = NT == 1 ? 36 * 1024 : 96 * 1024;

// 16 bytes to shared memory, zeros where !valid.
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 load_cached(const void* p) {
    uint4 r;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

__device__ __forceinline__ uint4 load_shared(uint32_t at) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at) : "memory");
    return r;
}

__device__ __forceinline__ uint32_t load_shared_word(uint32_t at) {
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
    return r;
}

// E2M1 codes p and p + 4 of a word (pair p = 0 .. 3) as bf16 times 2^-126: the
// sign to bit 15, exponent and mantissa to bits 6-8, where bf16's two lowest
// exponent values read E2M1's, zero and its subnormal included.  One product
// places both copies of the nibble (no carry: they do not overlap).
template <int PAIR>
__device__ __forceinline__ uint32_t spread(uint32_t w) {
    const uint32_t v = PAIR < 2 ? w : w >> 8;
    const uint32_t t = (PAIR & 1) ? (v & 0x00F000F0u) * 0x0104u : (v & 0x000F000Fu) * 0x1040u;
    return t & 0x81C081C0u;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if (F16) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
        return;
    }
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr uint32_t kTwo119 = 0x7B007B00u, kTwo120 = 0x7B807B80u;   // bf16 pairs

// The same in FP16, started from zero.
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%10, %10, %10, %10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Scales of a lane's 32 k of one feature.
//   NVFP4: two blocks; e4m3 times 2^119 as bf16 pairs.  A byte moved to bf16's
//     exponent and mantissa reads as the scale times 2^-120 (subnormals too);
//     0x7F, which would read as 480, is set to NaN.
//   MX: one block; 2^(byte - 1), or 2^127 and the rest in `over`.
template <bool MX>
struct Scales {
    uint32_t s[2];
    uint32_t over;
    __device__ __forceinline__ void set(uint32_t word, int t) {
        if (MX) {
            const uint32_t b = (word >> (8 * t)) & 0xFFu;
            const uint32_t lo = b < 128u ? b : 128u;
            s[0] = s[1] = ((lo + 126u) << 7) * 0x10001u;
            over = ((b - lo + 127u) << 7) * 0x10001u;
        } else {
            const uint32_t h = word >> (16 * (t & 1));
            uint32_t v;
            asm("prmt.b32 %0, %1, 0, 0x4140;" : "=r"(v) : "r"(h & 0x7F7Fu));
            v = mul_bf16x2(mul_bf16x2(v << 4, kTwo120), kTwo119) | (__vcmpeq2(v, 0x007F007Fu) & 0x7FFF7FFFu);
            asm("prmt.b32 %0, %1, 0, 0x1010;" : "=r"(s[0]) : "r"(v));
            asm("prmt.b32 %0, %1, 0, 0x3232;" : "=r"(s[1]) : "r"(v));
        }
    }
};

// The eight E2M1 codes of a word as FP16 pairs, in order.
__device__ __forceinline__ void decode_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// One item in FP16.  NVFP4: weights times their scales, added to acc.
template <int NT>
__device__ __forceinline__ void item_f16_nvfp4(const Item& it, const uint8_t* const (&xrow)[NT], int t, float (&acc)[2][NT][4]) {
    uint32_t sc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        const uint16_t two = (uint16_t)((word_of(it.sf, i) >> (16 * (t & 1))) & 0x7F7Fu);
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        sc[i][0] = __byte_perm(h, 0, 0x1010);
        sc[i][1] = __byte_perm(h, 0, 0x3232);
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint4 b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) b[j] = *reinterpret_cast<const uint4*>(xrow[j] + w * 64 + t * 16);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t f[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                decode_f16(word_of(it.codes[2 * u + i], w), f[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[i][e] = mul_f16x2(f[i][e], sc[2 * u + i][w >> 1]);
            }
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    mma<true>(acc[u][j], f[0][2 * half], f[1][2 * half], f[0][2 * half + 1], f[1][2 * half + 1], half ? b[j].z : b[j].x,
                              half ? b[j].w : b[j].y);
        }
    }
}

// One item of one row in FP16, NVFP4: the eight columns of B hold the row's eight blocks, each lane column's 32 k its
// two (zeros elsewhere), so a product's sums come apart by block and the scales are applied to them in FP32.
__device__ __forceinline__ void item_f16_one(const Item& it, const uint8_t* xrow, int g, int t, float (&acc)[4]) {
    float sum[2][4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint4 b = make_uint4(0, 0, 0, 0);
        if (g == t + 4 * (w >> 1)) b = *reinterpret_cast<const uint4*>(xrow + w * 64 + t * 16);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t f[2][4];
            decode_f16(word_of(it.codes[2 * u], w), f[0]);
            decode_f16(word_of(it.codes[2 * u + 1], w), f[1]);
            if (w == 0) mma_first(sum[u], f[0][0], f[1][0], f[0][1], f[1][1], b.x, b.y);
            else mma<true>(sum[u], f[0][0], f[1][0], f[0][1], f[1][1], b.x, b.y);
            mma<true>(sum[u], f[0][2], f[1][2], f[0][3], f[1][3], b.z, b.w);
        }
    }
    // columns 2 t and 2 t + 1: blocks 0 2, 4 6, 1 3, 5 7 (the lane's scale words are of the atom with its two)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        const uint16_t two = (uint16_t)(__byte_perm(word_of(it.sf, i), 0, t < 2 ? 0x4420 : 0x4431) & 0x7F7Fu);
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        const float2 s = __half22float2(*reinterpret_cast<const __half2*>(&h));
        acc[i] = fmaf(sum[i >> 1][2 * (i & 1)], s.x, acc[i]);
        acc[i] = fmaf(sum[i >> 1][2 * (i & 1) + 1], s.y, acc[i]);
    }
}

// One item in FP16, MX: a block's 32 k are one 16-byte piece of a feature, of which lane t takes word t, so that a
// product's sums are of one block and its scale is applied to them in FP32.  Pieces lie in the
// order the copies gave them: (4 g + (block ^ (g / 2 & 3))) 16 bytes into the feature's 512.
// SAFE: the rows' powers of two are undone first (see below).
template <int NT, bool SAFE>
__device__ __forceinline__ void item_f16_mx(uint32_t item, const uint4& sf, const uint8_t* const (&xrow)[NT], int g, int t,
                                            const float (&undo)[NT][2], float (&acc)[2][NT][4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint4 b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) b[j] = *reinterpret_cast<const uint4*>(xrow[j] + c * 64 + t * 16);
        const uint32_t at = item + (4 * g + (c ^ ((g >> 1) & 3))) * 16 + 4 * t;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t f[2][4];
            float s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                decode_f16(load_shared_word(at + (2 * u + i) * 512), f[i]);
                const uint32_t word = word_of(sf, 2 * u + i);
                if (SAFE) {                         // 2^(byte - 128), so that 2^128 is not needed
                    const uint32_t e = (word >> (8 * c)) & 0xFFu;
                    s[i] = __uint_as_float(e > 1u ? (e - 1u) << 23 : 0x00200000u << e);
                } else {                            // 2^(byte - 127)
                    s[i] = __uint_as_float(max((c < 3 ? word << (23 - 8 * c) : word >> 1) & 0x7F800000u, 0x00400000u));
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float sum[4];
                mma_first(sum, f[0][0], f[1][0], f[0][1], f[1][1], b[j].x, b[j].y);
                mma<true>(sum, f[0][2], f[1][2], f[0][3], f[1][3], b[j].z, b[j].w);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[u][j][e] = fmaf(SAFE ? sum[e] * undo[j][e & 1] : sum[e], s[e >> 1], acc[u][j][e]);
            }
        }
    }
}

// Out of line: nothing of it stays in registers where it is not called.
template <int NT>
__device__ __noinline__ void item_f16_mx_safe(uint32_t item, const uint4* sf, const uint8_t* const* xrow, int g, int t,
                                              const float* back, float* sums) {
    const uint8_t* xr[NT];
    float undo[NT][2], acc[2][NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) xr[j] = xrow[j];
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) (&undo[0][0])[i] = back[i];
#pragma unroll
    for (int i = 0; i < 8 * NT; ++i) (&acc[0][0][0])[i] = sums[i];
    item_f16_mx<NT, true>(item, *sf, xr, g, t, undo, acc);
#pragma unroll
    for (int i = 0; i < 8 * NT; ++i) sums[i] = (&acc[0][0][0])[i];
}

// One item in bf16: x pairs in the order (0,4) (1,5) (2,6) (3,7) of a code word.
template <int NT, bool MX>
__device__ __noinline__ void item_bf16(const Item* from, const uint8_t* const* xrow, int t, float* sums) {
    const Item it = *from;
    float acc[2][NT][4];
#pragma unroll
    for (int i = 0; i < 8 * NT; ++i) (&acc[0][0][0])[i] = sums[i];
    Scales<MX> sc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i].set(word_of(it.sf, i), t);
    const bool over =
        MX && __any_sync(0xffffffffu, ((sc[0].over | sc[1].over | sc[2].over | sc[3].over) & 0x7FFFu) != 0x3F80u);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint4 b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) b[j] = *reinterpret_cast<const uint4*>(xrow[j] + (MX ? t * 64 + w * 16 : w * 64 + t * 16));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t f[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t c = word_of(it.codes[i], w);
                const uint32_t sv = sc[i].s[w >> 1];
                f[i][0] = mul_bf16x2(half ? spread<2>(c) : spread<0>(c), sv);
                f[i][1] = mul_bf16x2(half ? spread<3>(c) : spread<1>(c), sv);
                if (over) {
                    f[i][0] = mul_bf16x2(f[i][0], sc[i].over);
                    f[i][1] = mul_bf16x2(f[i][1], sc[i].over);
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint32_t b0 = half ? b[j].z : b[j].x, b1 = half ? b[j].w : b[j].y;
                mma<false>(acc[0][j], f[0][0], f[1][0], f[0][1], f[1][1], b0, b1);
                mma<false>(acc[1][j], f[2][0], f[3][0], f[2][1], f[3][1], b0, b1);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8 * NT; ++i) sums[i] = (&acc[0][0][0])[i];
}

// ONE: a single row.
template <int NT, bool MX, bool ONE>
__global__ void __launch_bounds__(kThreads, 1) gemv_kernel(const Params p) {
    constexpr int kAhead = kDepth<NT>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint32_t x_max[16], x_min[16];               // of a row's k range: largest |x|, smallest nonzero |x| - 1, as bits
    __shared__ int head_unit[kWarps];                       // the unit a warp starts inside of, or -1
    constexpr int kEarly = 2;                               // pieces of x a thread loads before the first weights

    const GemvArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rank = (int)cluster_ctarank(), ranks = gridDim.y;
    const int c = blockIdx.x;
    const int u_first = c * p.units_each + min(c, p.units_more), u_last = u_first + p.units_each + (c < p.units_more ? 1 : 0);
    const int k_first = rank * p.steps_each + min(rank, p.steps_more), k_last = k_first + p.steps_each + (rank < p.steps_more ? 1 : 0);
    const int row_bytes = p.segment * 256 + 64;
    // this warp's items [slot][5][32] of 16 bytes, and this lane's place in them (MX: swizzled, see item_f16_mx)
    const uint32_t items = smem_u32(smem) + warp * kAhead * kItemBytes;
    const uint32_t ring = items + (MX ? 4 * g + (t ^ ((g >> 1) & 3)) : lane) * 16;
    uint8_t* const xs = smem + kWarps * kAhead * kItemBytes;    // [M][segment][4][4] 16-byte pieces of x (+ 64 bytes a row)
    float* const part = reinterpret_cast<float*>(xs + a.M * row_bytes);      // [unit_chunk][M][32]: sums
    float* const heads = part + p.unit_chunk * kUnitN * a.M;                   // [warp][M][32]: sums of units begun by another warp
    const int unit_floats = kUnitN * a.M;
    const int64_t row_codes = a.K / 2;

    const uint8_t* xrow[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) xrow[j] = xs + (ONE ? 0 : min(8 * j + g, a.M - 1)) * row_bytes;

    for (int u0 = u_first; u0 < u_last; u0 += p.unit_chunk) {
        const int units = min(p.unit_chunk, u_last - u0);
        for (int k0 = k_first; k0 < k_last; k0 += p.segment) {
            const int steps = min(p.segment, k_last - k0);
            const int total = units * steps;
            int item = total / kWarps * warp + min(warp, total % kWarps);
            const int end = item + total / kWarps + (warp < total % kWarps ? 1 : 0);

            // the next items' weights
            int fu = item / steps, fk = item - fu * steps, left = end - item;
            const uint8_t *codes = nullptr, *sf = nullptr;
            uint32_t have = 0;
            auto aim = [&]() {
                const int u = u0 + fu, n = (u >> 2) * 128 + (u & 3) * 8 + g;
                have = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) have |= (n + 32 * i < a.N ? 1u : 0u) << i;
                codes = a.w_codes + (int64_t)n * row_codes + 16 * t;
                sf = a.w_sf + (int64_t)(u >> 2) * p.kb4 * 512 + ((u & 3) * 8 + g) * 16;
            };
            auto fetch = [&](int slot) {
                if (left <= 0) {
                    copies_commit();
                    return;
                }
                const int s = k0 + fk;
                const bool in = s * kStepK + 32 * t < a.K;  // a last half step has no k for t >= 2
                const uint32_t dst = ring + slot * kItemBytes;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool valid = in && (have >> i & 1u);
                    copy_async(dst + i * 512, valid ? codes + i * 32 * row_codes + (int64_t)s * 64 : a.w_codes, valid);
                }
                // scales: of the lane's own blocks, or (ONE) of the atom with its columns' blocks
                const int atom = MX ? s : 2 * s + (ONE ? t & 1 : t >> 1);
                const bool has = atom < p.kb4;
                copy_async(dst + 4 * 512, has ? sf + (int64_t)atom * 512 : a.w_sf, has);
                copies_commit();
                --left;
                if (++fk == steps) {
                    fk = 0;
                    ++fu;
                    if (left > 0) aim();
                }
            };
            // x of the k range (several warps a row, or several rows a warp), its first loads ahead of the weights'
            const int per_row = max(1, kWarps / a.M), pieces = steps * 16;     // warps of a row
            const int p_first = (warp % per_row) * 32 + lane, p_step = per_row * 32;
            const int m_first = warp / per_row, m_step = kWarps / per_row;
            auto piece = [&](int m, int q) {
                return reinterpret_cast<uint4*>(xs + m * row_bytes + (q >> 4) * 256 + (MX ? (q & 15) * 16 : (q & 3) * 64 + ((q >> 2) & 3) * 16));
            };
            auto load_x = [&](int m, int q) {
                const int k = k0 * kStepK + q * 8;
                return q < pieces && k < a.K ? load_cached(a.x + (int64_t)m * a.ld_x + k) : make_uint4(0, 0, 0, 0);
            };
            uint4 early[kEarly];
#pragma unroll
            for (int i = 0; i < kEarly; ++i) early[i] = m_first < a.M ? load_x(m_first, p_first + i * p_step) : make_uint4(0, 0, 0, 0);
            int unit = fu, step = fk;
            const bool begins = fk == 0, some = item < end;
            if (left > 0) aim();
#pragma unroll
            for (int i = 0; i < kAhead; ++i) fetch(i);

            if (u0 != u_first || k0 != k_first) __syncthreads();
            if (threadIdx.x < 16) {
                x_max[threadIdx.x] = 0;
                x_min[threadIdx.x] = 0xFFFFu;
            }
            if (lane == 0) head_unit[warp] = some && !begins ? unit : -1;
            __syncthreads();
            for (int m = m_first; m < a.M; m += m_step) {
                uint32_t hi = 0, lo = 0xFFFFFFFFu;
                auto take = [&](int q, const uint4& v) {
                    *piece(m, q) = v;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t b = word_of(v, i) & 0x7FFF7FFFu;
                        hi = __vmaxu2(hi, b);
                        lo = __vminu2(lo, __vsub2(b, 0x00010001u));
                    }
                };
                int q = p_first;
                if (m == m_first)
#pragma unroll
                    for (int i = 0; i < kEarly; ++i, q += p_step)
                        if (q < pieces) take(q, early[i]);
                constexpr int kBatch = 5;
                for (; q < pieces; q += kBatch * p_step) {
                    uint4 v[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) v[i] = load_x(m, q + i * p_step);
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        if (q + i * p_step < pieces) take(q + i * p_step, v[i]);
                }
                hi = __reduce_max_sync(0xffffffffu, max(hi & 0xFFFFu, hi >> 16));
                lo = __reduce_min_sync(0xffffffffu, min(lo & 0xFFFFu, lo >> 16));
                if (lane == 0) {
                    atomicMax(&x_max[m], hi);
                    atomicMin(&x_min[m], lo);
                }
            }
            __syncthreads();
            bool fits = true;                               // every row within FP16's exact range
            for (int i = 0; i < a.M; ++i) {
                const int top = (int)(x_max[i] >> 7), low = (int)((x_min[i] + 1) >> 7);
                fits = fits && (x_max[i] == 0 || (top >= 64 && top <= (MX ? 141 : 190) && low >= top - 31));
            }
            for (int m = m_first; m < a.M; m += m_step) {
                const int top = (int)(x_max[m] >> 7);
                const float by = x_max[m] ? __uint_as_float((uint32_t)(127 + 14 + 127 - top) << 23) : 1.0f;
                for (int q = p_first; q < pieces; q += p_step) {
                    const uint4 v = *piece(m, q);
                    uint32_t o[4];
                    if (fits) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t w = word_of(v, i);
                            const __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * by, __uint_as_float(w & 0xFFFF0000u) * by);
                            o[i] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                    } else {
                        o[0] = __byte_perm(v.x, v.z, 0x5410);
                        o[1] = __byte_perm(v.x, v.z, 0x7632);
                        o[2] = __byte_perm(v.y, v.w, 0x5410);
                        o[3] = __byte_perm(v.y, v.w, 0x7632);
                    }
                    *piece(m, q) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            __syncthreads();

            float undo[NT][2];                              // of this lane's rows' powers of two
#pragma unroll
            for (int i = 0; i < 2 * NT; ++i) {
                const uint32_t top = x_max[8 * (i >> 1) + 2 * t + (i & 1)] >> 7;
                undo[i >> 1][i & 1] = fits && top ? __uint_as_float((top - 14u) << 23) : 1.0f;
            }
            float acc[2][NT][4] = {}, one[4] = {};
            bool first_unit = true, raised = false;
            auto flush = [&]() {                            // sums of the unit, in units of x and the weights
                const bool head = first_unit && !begins;
                float* dst = head ? heads + warp * unit_floats : part + unit * unit_floats;
                const bool add = !head && k0 != k_first;
                if (ONE && fits) {                          // a lane's columns are blocks: their sum is the row's
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        one[i] += __shfl_xor_sync(0xffffffffu, one[i], 1);
                        one[i] += __shfl_xor_sync(0xffffffffu, one[i], 2);
                        acc[i >> 1][0][2 * (i & 1)] = one[i];
                        one[i] = 0.0f;
                    }
                }
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int row = 8 * j + 2 * t + c;
                        if (row >= a.M) continue;
                        // the bf16 path's NVFP4 weights are 2^-7 of theirs, E8M0 scales of raised units half of theirs
                        const float by = fits ? (MX ? (raised ? 2.0f : undo[j][c]) : undo[j][c]) : (MX ? 1.0f : 128.0f);
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float* at = dst + row * kUnitN + 8 * (2 * u + h) + g;
                                const float v = acc[u][j][2 * h + c] * by;
                                *at = add ? *at + v : v;
                                acc[u][j][2 * h + c] = 0.0f;
                            }
                    }
                first_unit = false;
                raised = false;
            };
            auto run = [&](Item& it, uint32_t at) {
                const uint8_t* xr[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) xr[j] = xrow[j] + step * 256;
                if (MX && fits && !raised) {
                    // Scales above 2^90 could leave FP32's range with the rows' powers of two: from such an item on, the
                    // unit's sums are kept without them.
                    const uint32_t m = __vmaxu4(__vmaxu4(it.sf.x, it.sf.y), __vmaxu4(it.sf.z, it.sf.w));
                    raised = __any_sync(0xffffffffu, __vcmpgtu4(m, 0xD9D9D9D9u) != 0u);
                    if (raised)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int j = 0; j < NT; ++j)
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[u][j][e] *= 0.5f * undo[j][e & 1];
                }
                if (!fits || raised) {
                    Item copy = it;
                    if (ONE) {                              // the scales of the lane's own blocks, from a lane that has them
                        const int from = (lane & ~3) | (t >> 1);
                        copy.sf = make_uint4(__shfl_sync(0xffffffffu, it.sf.x, from), __shfl_sync(0xffffffffu, it.sf.y, from),
                                             __shfl_sync(0xffffffffu, it.sf.z, from), __shfl_sync(0xffffffffu, it.sf.w, from));
                    }
                    float sums[8 * NT], back[2 * NT];
#pragma unroll
                    for (int i = 0; i < 8 * NT; ++i) sums[i] = (&acc[0][0][0])[i];
#pragma unroll
                    for (int i = 0; i < 2 * NT; ++i) back[i] = (&undo[0][0])[i];
                    if (!fits) item_bf16<NT, MX>(&copy, xr, t, sums);
                    else if (MX) item_f16_mx_safe<NT>(at, &copy.sf, xr, g, t, back, sums);
#pragma unroll
                    for (int i = 0; i < 8 * NT; ++i) (&acc[0][0][0])[i] = sums[i];
                } else if (MX) {
                    item_f16_mx<NT, false>(at, it.sf, xr, g, t, undo, acc);
                } else if (ONE) {
                    item_f16_one(it, xr[0], g, t, one);
                } else {
                    item_f16_nvfp4<NT>(it, xr, t, acc);
                }
                ++item;
                if (++step == steps) {
                    flush();
                    step = 0;
                    ++unit;
                }
            };
            for (int slot = 0; item < end; slot = slot + 1 == kAhead ? 0 : slot + 1) {
                copies_wait<kAhead - 1>();                  // a lane reads what it copied itself; MX: what the warp did
                if (MX) __syncwarp();
                Item it;
                auto load_codes = [&]() {
#pragma unroll
                    for (int i = 0; i < 4; ++i) it.codes[i] = load_shared(ring + slot * kItemBytes + i * 512);
                };
                if (!MX || !fits) load_codes();             // item_f16_mx reads them where they are
                it.sf = load_shared(ring + slot * kItemBytes + 4 * 512);
                run(it, items + slot * kItemBytes);
                if (MX) __syncwarp();                       // before the slot is filled again
                fetch(slot);
            }
            copies_wait<0>();
            if (some && step != 0) flush();
            __syncthreads();
            // what warps added to units that another one began, in the warps' order; a warp takes every kWarps-th unit
            for (int w = 1; w < kWarps; ++w) {
                const int u = head_unit[w];
                if (u < 0 || u % kWarps != warp) continue;
                for (int i = lane; i < unit_floats; i += 32) part[u * unit_floats + i] += heads[w * unit_floats + i];
            }
        }
        if (ranks > 1) cluster_sync_all();
        else __syncthreads();
        // the blocks' sums, in rank order; each block finishes a part of the features
        const float scale = a.w_scale ? __ldg(a.w_scale) : 1.0f;
        const int floats = units * unit_floats;
        const int share = (floats + ranks - 1) / ranks, f_first = share * rank, f_last = min(f_first + share, floats);
        for (int i = f_first + threadIdx.x; i < f_last; i += kThreads) {
            const int u = i / unit_floats, r = i - u * unit_floats, row = r / kUnitN, f = r & (kUnitN - 1);
            const int n = ((u0 + u) >> 2) * 128 + ((u0 + u) & 3) * 8 + (f >> 3) * 32 + (f & 7);
            float v = 0.0f;
            if (ranks > 1) {
                const uint32_t at = smem_u32(part + i);
                for (int q = 0; q < ranks; ++q) {
                    float x;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(mapa_shared(at, (uint32_t)q)));
                    v += x;
                }
            } else {
                v = part[i];
            }
            if (n < a.N) {
                v *= scale;
                if (a.bias) v += __ldg(a.bias + n);
                if (a.y_f32) static_cast<float*>(a.y)[(int64_t)row * a.N + n] = v;
                else static_cast<__nv_bfloat16*>(a.y)[(int64_t)row * a.N + n] = __float2bfloat16_rn(v);
            }
        }
        if (ranks > 1) cluster_sync_all();                  // the others may still read this block's sums
    }
}

template <int NT, bool MX, bool ONE>
cudaError_t launch(const Params& p, int clusters, int ranks, int smem, cudaStream_t stream) {
    // always the same limit: it belongs to the kernel, and another thread may be about to launch with more
    cudaError_t e = cudaFuncSetAttribute(gemv_kernel<NT, MX, ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)clusters, (unsigned)ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1;
    attr.val.clusterDim.y = (unsigned)ranks;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = ranks > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, gemv_kernel<NT, MX, ONE>, p);
    if (e == cudaSuccess) count_launch(1);
    return e;
}

// Clusters of `ranks` blocks (one block an SM) that the device runs at once: asked for once per device.
int64_t resident_clusters(bool two, bool mx, int ranks, int num_sms) {
    if (ranks <= 2) return num_sms / ranks;
    static std::atomic<int> known[64][2];                   // for four, eight blocks
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
    std::atomic<int>& slot = known[dev][ranks == 8];
    int n = slot.load(std::memory_order_relaxed);
    if (n == 0) {
        const void* kernel = two ? (mx ? (const void*)gemv_kernel<2, true, false> : (const void*)gemv_kernel<2, false, false>)
                                 : (mx ? (const void*)gemv_kernel<1, true, false> : (const void*)gemv_kernel<1, false, false>);
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) != cudaSuccess) return 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)num_sms, (unsigned)ranks);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemLimit;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 1;
        attr.val.clusterDim.y = (unsigned)ranks;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
            (void)cudaGetLastError();
            return 1;
        }
        slot.store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace gemv

cudaError_t launch_gemv(const GemvArgs& a, int num_sms, cudaStream_t stream) {
    using namespace gemv;
    Params p{};
    p.a = a;
    p.units = (a.N + 127) / 128 * 4;
    p.steps = (a.K + kStepK - 1) / kStepK;
    p.kb4 = a.K / (a.mx ? 128 : 64);
    // Blocks along k: the number that ends first, in sixteenths of a round of items (one item of each warp); a cluster's
    // start and join cost about two rounds, and a block reads, scans and converts its part of x first, 128 k of a row
    // for a 9th of a sixteenth.  (Against each number by force, 6 shapes of both formats at 1, 4, 8 and 16 rows: the
    // choice is within 5 % of the best in 30 of these 48 and up to 1.5 times it in the rest, 4 rows of 5120 -> 5120
    // 18.5 us for 12.3.  There x costs more than the 9th: 0.03 us a row and 128 k, where a round takes 1.2 us at one row
    // and 2.4 at sixteen.)  The clusters all run at once: more of them than the GPCs hold would double the time.
    int ranks = 1, clusters = 1;
    int64_t best = 0;
    for (int r = 1; r <= kMaxCluster && r <= p.steps; r *= 2) {
        const int64_t most = resident_clusters(a.M > 8, a.mx, r, num_sms);
        const int64_t c = p.units < most ? p.units : most;
        const int64_t per = (p.units + c - 1) / c, steps = (p.steps + r - 1) / r;
        const int64_t cost = 16 * ((per * steps + kWarps - 1) / kWarps + (r > 1 ? 2 : 0)) + a.M * steps / 9;
        if (best == 0 || cost < best) {
            best = cost;
            ranks = r;
            clusters = (int)c;
        }
    }
    p.units_each = p.units / clusters;
    p.units_more = p.units % clusters;
    p.steps_each = p.steps / ranks;
    p.steps_more = p.steps % ranks;
    const int steps = (p.steps + ranks - 1) / ranks;
    const int unit_bytes = kUnitN * a.M * 4;
    // shared memory: the warps' items, x of a k segment, the warps' heads, the sums of as many units as are left room for
    const int ring_bytes = kWarps * kItemBytes * (a.M <= 8 ? kDepth<1> : kDepth<2>);
    p.segment = ((a.M <= 8 ? kXBytes<1> : kXBytes<2>) / a.M - 64) / 256;
    if (p.segment > steps) p.segment = steps;
    const int x_bytes = a.M * (p.segment * 256 + 64);
    const int per = (p.units + clusters - 1) / clusters;
    p.unit_chunk = (kSmemLimit - ring_bytes - x_bytes - kWarps * unit_bytes) / unit_bytes;
    if (p.unit_chunk > per) p.unit_chunk = per;
    const int smem = ring_bytes + x_bytes + (kWarps + p.unit_chunk) * unit_bytes;
    if (a.M <= 8)
        return a.mx       ? launch<1, true, false>(p, clusters, ranks, smem, stream)
               : a.M == 1 ? launch<1, false, true>(p, clusters, ranks, smem, stream)
                          : launch<1, false, false>(p, clusters, ranks, smem, stream);
    return a.mx ? launch<2, true, false>(p, clusters, ranks, smem, stream) : launch<2, false, false>(p, clusters, ranks, smem, stream);
}

}  // namespace nvfp4
