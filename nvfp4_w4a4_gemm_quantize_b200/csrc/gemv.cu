// gemv.cu -- a few rows of activations times 4-bit weights with group scales
// (nvfp4_gemv_w4a16):
//   y[m,n] = g sum_k x[m,k] e2m1(w[n,k]) s[n, k / block] (+ bias[n]),  M <= 16.
// Bound by reading the weights once, N K / 2 + N K / block bytes.
//
// The weights are the A operand of m16n8k16 products (16 output features, 8
// rows of x), so one decoded register serves every row of x.  A block has 128
// features (the rows of one scale atom group) and 8 warps: four over the
// features, two over k.  A lane holds features 32 i + 8 w + lane / 4 (i < 4),
// whose scales of 64 k are one 16-byte word of the scale layout, and of each
// 128 k reads 16 code bytes a feature, 32 neighbouring k: the order of k within
// a product is free as long as x comes in the same one, so nothing is shuffled.
// x is kept in shared memory in that order.
// The k range is split over the CTAs of a cluster (so that a matrix with few
// features still fills the SMs); their sums are added over distributed shared
// memory in rank order, so results do not depend on timing and need no workspace.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dit.h"
#include "internal.h"
#include "ptx.cuh"

namespace nvfp4 {
namespace gemv {

constexpr int kThreads = 256;
constexpr int kTileN = 128;                   // features of a block
constexpr int kWarpsK = 2;
constexpr int kStepK = 128;                   // k of a warp's step
constexpr int kMaxCluster = 8;
constexpr int kXBytes = 72 * 1024;            // x kept at a time

struct Params {
    GemvArgs a;
    int steps;                                // ceil(K / 128)
    int segment;                              // steps of x kept at a time
    int kb4;                                  // scale atoms along k: K / (4 block)
};

// One 128-k step of a lane: 16 code bytes and the scales of its four features.
struct Step {
    uint4 codes[4];
    uint4 sf;                                 // word i: four blocks of feature i
};

__device__ __forceinline__ uint4 load_stream(const void* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
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

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr uint32_t kTwo119 = 0x7B007B00u, kTwo120 = 0x7B807B80u;   // bf16 pairs

// Scales of a lane's 32 k of one feature.
//   NVFP4: two blocks; e4m3 times 2^119 as bf16 pairs.  A byte moved to bf16's
//     exponent and mantissa reads as the scale times 2^-120 (subnormals too).
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
            v = mul_bf16x2(mul_bf16x2(v << 4, kTwo120), kTwo119);
            asm("prmt.b32 %0, %1, 0, 0x1010;" : "=r"(s[0]) : "r"(v));
            asm("prmt.b32 %0, %1, 0, 0x3232;" : "=r"(s[1]) : "r"(v));
        }
    }
};

// Weights are kept times this power of two until the sums are complete.
template <bool MX>
constexpr float kUndo = MX ? 1.0f : 128.0f;

template <int NT, bool MX>
__global__ void __launch_bounds__(kThreads, 2) gemv_kernel(const Params p) {
    extern __shared__ __align__(16) uint8_t xs[];           // [M][segment][4][4] 16-byte pieces of x (+ 64 bytes a row)
    __shared__ float part[NT * 8][kTileN];                  // this CTA's sums

    const GemvArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int wn = warp & 3, wk = warp >> 2;
    const int rank = (int)cluster_ctarank(), ranks = gridDim.y;
    const int nb = blockIdx.x;
    const int first = (int)((int64_t)p.steps * rank / ranks), last = (int)((int64_t)p.steps * (rank + 1) / ranks);
    const int row_bytes = p.segment * 256 + 64;

    // this lane's features and, within a step, its 32 k
    const uint8_t* codes[4];
    uint32_t have = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = nb * kTileN + 32 * i + 8 * wn + g;
        have |= (n < a.N ? 1u : 0u) << i;
        codes[i] = a.w_codes + (int64_t)(n < a.N ? n : 0) * (a.K / 2) + 16 * t;
    }
    const uint8_t* sf = a.w_sf + (int64_t)nb * p.kb4 * 512 + (8 * wn + g) * 16;
    auto fetch = [&](int s, Step& st) {
        const bool in = s < last && s * kStepK + 32 * t < a.K;      // a last half step has no k for t >= 2
#pragma unroll
        for (int i = 0; i < 4; ++i)
            st.codes[i] = in && (have >> i & 1u) ? load_stream(codes[i] + (int64_t)s * 64) : make_uint4(0, 0, 0, 0);
        st.sf = in ? load_stream(sf + (int64_t)(MX ? s : 2 * s + (t >> 1)) * 512) : make_uint4(0, 0, 0, 0);
    };

    float acc[2][NT][4] = {};
    Step cur, nxt;
    int s = first + wk;
    fetch(s, cur);
    const uint8_t* xrow[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) xrow[j] = xs + min(8 * j + g, a.M - 1) * row_bytes + t * 16;

    for (int seg = first; seg < last; seg += p.segment) {
        const int seg_end = min(seg + p.segment, last);
        if (seg != first) __syncthreads();
        // x of the segment, eight values a piece in the order (0,4) (1,5) (2,6) (3,7) of a code word;
        // piece i of lane column t of a step sits at i * 64 + t * 16 (conflict-free reads)
        const int pieces = (seg_end - seg) * 16;
        for (int i = threadIdx.x; i < pieces * a.M; i += kThreads) {
            const int m = i / pieces, q = i - m * pieces, k = seg * kStepK + q * 8;
            uint4 v = make_uint4(0, 0, 0, 0), o;
            if (k < a.K) v = __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)m * a.ld_x + k));
            o.x = __byte_perm(v.x, v.z, 0x5410);
            o.y = __byte_perm(v.x, v.z, 0x7632);
            o.z = __byte_perm(v.y, v.w, 0x5410);
            o.w = __byte_perm(v.y, v.w, 0x7632);
            *reinterpret_cast<uint4*>(xs + m * row_bytes + (q >> 4) * 256 + (q & 3) * 64 + ((q >> 2) & 3) * 16) = o;
        }
        __syncthreads();
        for (; s < seg_end; s += kWarpsK) {
            fetch(s + kWarpsK, nxt);
            Scales<MX> sc[4];
            const uint32_t sfw[4] = {cur.sf.x, cur.sf.y, cur.sf.z, cur.sf.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[i].set(sfw[i], t);
            const bool over = MX && __any_sync(0xffffffffu, ((sc[0].over | sc[1].over | sc[2].over | sc[3].over) & 0x7FFFu) != 0x3F80u);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint4 b[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) b[j] = *reinterpret_cast<const uint4*>(xrow[j] + (s - seg) * 256 + w * 64);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t f[4][2];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t c = w == 0 ? cur.codes[i].x : w == 1 ? cur.codes[i].y : w == 2 ? cur.codes[i].z : cur.codes[i].w;
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
                        mma(acc[0][j], f[0][0], f[1][0], f[0][1], f[1][1], b0, b1);
                        mma(acc[1][j], f[2][0], f[3][0], f[2][1], f[3][1], b0, b1);
                    }
                }
            }
            cur = nxt;
        }
    }

    // the two k halves of the block, then the cluster's CTAs, in a fixed order
#pragma unroll
    for (int h = kWarpsK - 1; h >= 0; --h) {
        if (wk == h) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float* d = &part[8 * j + 2 * t + (e & 1)][32 * (2 * u + (e >> 1)) + 8 * wn + g];
                        *d = h == kWarpsK - 1 ? acc[u][j][e] : *d + acc[u][j][e];
                    }
        }
        __syncthreads();
    }
    if (ranks > 1) cluster_sync_all();
    const float scale = (a.w_scale ? __ldg(a.w_scale) : 1.0f) * kUndo<MX>;
    const int share = kTileN / ranks;                       // features this CTA finishes
    for (int i = threadIdx.x; i < share * a.M; i += kThreads) {
        const int m = i / share, c = rank * share + i - m * share, n = nb * kTileN + c;
        const uint32_t at = smem_u32(&part[m][c]);
        float v = 0.0f;
        for (int r = 0; r < ranks; ++r) {
            float q;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(q) : "r"(mapa_shared(at, (uint32_t)r)));
            v += q;
        }
        if (n < a.N) {
            v *= scale;
            if (a.bias) v += __ldg(a.bias + n);
            if (a.y_f32) static_cast<float*>(a.y)[(int64_t)m * a.N + n] = v;
            else static_cast<__nv_bfloat16*>(a.y)[(int64_t)m * a.N + n] = __float2bfloat16_rn(v);
        }
    }
    if (ranks > 1) cluster_sync_all();                      // the others may still read this CTA's sums
}

template <int NT, bool MX>
cudaError_t launch(const Params& p, int blocks, int ranks, int smem, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(gemv_kernel<NT, MX>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1;
    attr.val.clusterDim.y = (unsigned)ranks;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, gemv_kernel<NT, MX>, p);
    if (e == cudaSuccess) count_launch(1);
    return e;
}

}  // namespace gemv

cudaError_t launch_gemv(const GemvArgs& a, int num_sms, cudaStream_t stream) {
    using namespace gemv;
    Params p{};
    p.a = a;
    p.steps = (a.K + kStepK - 1) / kStepK;
    p.kb4 = a.K / (a.mx ? 128 : 64);
    const int blocks = (a.N + kTileN - 1) / kTileN;
    // as many CTAs along k as leave every warp a step, until the SMs hold four blocks each
    int ranks = 1;
    while (ranks < kMaxCluster && p.steps >= 2 * ranks * kWarpsK && blocks * ranks < 4 * num_sms) ranks *= 2;
    const int per_rank = (p.steps + ranks - 1) / ranks;
    p.segment = (kXBytes / a.M - 64) / 256;
    if (p.segment > per_rank) p.segment = per_rank;
    // whole rounds of the block's warps, so that each warp's next step stays its own
    if (p.segment > kWarpsK) p.segment -= p.segment % kWarpsK;
    const int smem = a.M * (p.segment * 256 + 64);
    if (a.M <= 8)
        return a.mx ? launch<1, true>(p, blocks, ranks, smem, stream) : launch<1, false>(p, blocks, ranks, smem, stream);
    return a.mx ? launch<2, true>(p, blocks, ranks, smem, stream) : launch<2, false>(p, blocks, ranks, smem, stream);
}

}  // namespace nvfp4
