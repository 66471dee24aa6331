// xattn_few.cu -- attention of a few queries to an encoder's states
// (nvfp4_cross_attention with at most 16 rows, queries x heads that share a key /
// value head): the form for single tokens.
//
// Bound by reading K and V once.  The rows are the A operand of m16n8k16 products,
// S = Q K^T and O += P V, with an online softmax in registers (P goes from the
// first product's sums to the second's A operand without leaving the lane, rounded
// to bf16 as V is: the output is 2.1e-3 off the formula in 64 bits, in the norm,
// where FP32 arithmetic rounded once is 1.7e-3).
// Every warp is a stream of its own over a range of the keys: it loads slices of
// 32 keys of K and V by TMA into a ring of its own and refills a slot when it has
// used it, so nothing in the loop waits for another warp.  The keys of a (sample,
// key / value head) are split over the warps of a block and the blocks of a
// cluster; their (maximum, sum, O) are joined in a fixed order, warps over shared,
// blocks over distributed shared memory, without a workspace.
// B200, 8 samples' single token over 750 to 1500 states, 16 heads of 64 (43.7 MB):
// 14 us, of which the first loads' latency and the joins take about half.
#include "xattn.cuh"

namespace nvfp4 {
namespace xattn {

// Warps of a block: their rings fill most of an SM's shared memory.
template <int DS>
constexpr int kWarpsOf = DS == 4 ? 8 : 4;
constexpr int kSlice = 32;                    // keys of a slice
constexpr int kSliceChunk = kSlice * 128;     // bytes of 64 of its columns
constexpr int kFewStages = 3;
constexpr int kFewRows = 16;
constexpr int kFewMaxCluster = 8;

struct FewParams {
    MapAxes ak, av;
    nvfp4_heads q, out;
    float* lse;
    const int32_t* kv_lens;
    float c;                                  // scale * log2(e)
    int H, Hkv, Lq, Lk, d, group, chunks;
    int* dev_status;
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_m16n8k16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// DS: steps of 16 columns kept in registers, at least ceil(d / 16).
template <int DS>
__global__ void __launch_bounds__(32 * kWarpsOf<DS>)
xattn_few_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v, const FewParams p) {
    constexpr int kFewWarps = kWarpsOf<DS>, kFewThreads = 32 * kFewWarps;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kFewWarps][kFewStages];
    __shared__ float ms[kFewWarps][kFewRows], ls[kFewWarps][kFewRows];     // the warps' maxima (scaled, base 2) and sums
    __shared__ float bm[kFewRows], bl[kFewRows];                           // the block's
    __shared__ int abort_sh;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rank = (int)cluster_ctarank(), ranks = gridDim.y;
    const int b = blockIdx.x / p.Hkv, hk = blockIdx.x - b * p.Hkv, rows = p.group * p.Lq;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int slice_bytes = p.chunks * kSliceChunk, stage_bytes = 2 * slice_bytes;
    uint8_t* ring = smem + warp * kFewStages * stage_bytes;
    WaitCtx wc{&abort_sh, p.dev_status};

    // this warp's slices
    const int keys = keys_of(p.kv_lens, b, p.Lk);
    const int slices = (keys + kSlice - 1) / kSlice, streams = ranks * kFewWarps, stream = rank * kFewWarps + warp;
    const int each = slices / streams, more = slices - each * streams;
    const int first = stream * each + min(stream, more), last = first + each + (stream < more ? 1 : 0);

    if (threadIdx.x == 0) abort_sh = 0;
    if (lane == 0) {
        for (int i = 0; i < kFewStages; ++i) mbar_init(&full[warp][i], 1);
        fence_barrier_init();
    }
    __syncthreads();
    auto load = [&](int s, int stage) {             // by lane 0
        uint8_t* dst = ring + stage * stage_bytes;
        mbar_arrive_expect_tx(&full[warp][stage], (uint32_t)stage_bytes);
        load_tile(dst, &tmap_k, &full[warp][stage], p.chunks, kSliceChunk, hk * p.ak.h, s * kSlice, b * p.ak.b);
        load_tile(dst + slice_bytes, &tmap_v, &full[warp][stage], p.chunks, kSliceChunk, hk * p.av.h, s * kSlice, b * p.av.b);
    };
    if (lane == 0)
        for (int i = 0; i < kFewStages && first + i < last; ++i) load(first + i, i);

    // rows g and g + 8 of Q as A operands
    uint32_t qa[DS][4];
    const uint16_t* q_row[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int r = g + 8 * u, h = r / p.Lq, l = r - h * p.Lq;
        q_row[u] = r < rows ? static_cast<const uint16_t*>(p.q.data) + (int64_t)b * p.q.batch_stride + (int64_t)l * p.q.token_stride +
                                  (int64_t)(hk * p.group + h) * p.q.head_stride
                            : nullptr;
    }
#pragma unroll
    for (int kk = 0; kk < DS; ++kk)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int col = kk * 16 + (e >> 1) * 8 + 2 * t;
            qa[kk][e] = q_row[e & 1] && col < p.d ? __ldg(reinterpret_cast<const uint32_t*>(q_row[e & 1] + col)) : 0u;
        }

    const int dsteps = (p.d + 15) >> 4;
    float o[2 * DS][4] = {};
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int s = first; s < last; ++s) {
        if (!(ok = warp_wait(&full[warp][stage], phase, wc))) break;
        uint8_t* tile = ring + stage * stage_bytes;
        const uint32_t kt = smem_u32(tile), vt = kt + slice_bytes;
        const int n = min(keys - s * kSlice, kSlice);
        if (n < kSlice && keys < p.Lk) {
            // values past the length meet P = 0, but may be NaN: zeros
            for (int i = lane; i < (kSlice - n) * 8 * p.chunks; i += 32) {
                const int c = i / ((kSlice - n) * 8), r = i - c * (kSlice - n) * 8;
                *reinterpret_cast<uint4*>(tile + slice_bytes + c * kSliceChunk + n * 128 + r * 16) = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
        }
        float sc[4][4] = {};
#pragma unroll
        for (int kk = 0; kk < DS; ++kk) {
            if (kk >= dsteps) break;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t r[4];
                const int row = half * 16 + (lane >> 4) * 8 + (lane & 7), c16 = kk * 2 + ((lane >> 3) & 1);
                ldmatrix_x4(r, kt + (c16 >> 3) * kSliceChunk + row * 128 + (((c16 & 7) ^ (row & 7)) << 4));
                mma_m16n8k16(sc[2 * half], qa[kk], r[0], r[1]);
                mma_m16n8k16(sc[2 * half + 1], qa[kk], r[2], r[3]);
            }
        }
        if (n < kSlice) {
            // keys past the length: -infinity whatever was computed there
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j * 8 + 2 * t + (e & 1) >= n) sc[j][e] = -INFINITY;
        }
        float alpha[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float mx = fmaxf(fmaxf(fmaxf(sc[0][2 * u], sc[0][2 * u + 1]), fmaxf(sc[1][2 * u], sc[1][2 * u + 1])),
                             fmaxf(fmaxf(sc[2][2 * u], sc[2][2 * u + 1]), fmaxf(sc[3][2 * u], sc[3][2 * u + 1])));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * p.c;
            const float mn = fmaxf(m[u], mx);
            alpha[u] = mn > m[u] ? ex2(m[u] - mn) : 1.0f;
            m[u] = mn;
            const float mm = mn == -INFINITY ? 0.0f : -mn;           // all logits -infinity so far: P is 0, not NaN
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sc[j][2 * u + e] = ex2(fmaf(sc[j][2 * u + e], p.c, mm));
                    sum += sc[j][2 * u + e];
                }
            l[u] = fmaf(l[u], alpha[u], sum);
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
            for (int j = 0; j < 2 * DS; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][e] *= alpha[e >> 1];
        }
        uint32_t pa[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                pa[h][e] = pack_bf16(sc[2 * h + (e >> 1)][2 * (e & 1)], sc[2 * h + (e >> 1)][2 * (e & 1) + 1]);
#pragma unroll
        for (int kk = 0; kk < DS; ++kk) {
            if (kk >= dsteps) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t r[4];
                const int row = h * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), c16 = kk * 2 + (lane >> 4);
                ldmatrix_x4_trans(r, vt + (c16 >> 3) * kSliceChunk + row * 128 + (((c16 & 7) ^ (row & 7)) << 4));
                mma_m16n8k16(o[2 * kk], pa[h], r[0], r[1]);
                mma_m16n8k16(o[2 * kk + 1], pa[h], r[2], r[3]);
            }
        }
        __syncwarp();
        if (lane == 0 && s + kFewStages < last) load(s + kFewStages, stage);
        if (++stage == kFewStages) {
            stage = 0;
            phase ^= 1u;
        }
    }
    if (!ok && lane == 0) {                         // a warp that gave up still waits for its loads in flight
        int dummy = 0;
        WaitCtx w2{&dummy, p.dev_status};
        for (int i = 0; i < kFewStages; ++i) {
            mbar_wait_limit(&full[warp][stage], phase, w2, 1000000);
            if (++stage == kFewStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }

    // the warps' results: O to shared memory, over the rings
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
        if (t == 0) {
            ms[warp][g + 8 * u] = m[u];
            ls[warp][g + 8 * u] = l[u];
        }
    }
    __syncthreads();                                // no warp reads its ring any more
    const int pitch = DS * 16 + 8;                  // floats: rows of a quad's neighbours on other banks
    float* const os = reinterpret_cast<float*>(smem);                      // [warp][16][pitch]
#pragma unroll
    for (int j = 0; j < 2 * DS; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u)
            *reinterpret_cast<float2*>(os + (warp * kFewRows + g + 8 * u) * pitch + j * 8 + 2 * t) =
                make_float2(o[j][2 * u], o[j][2 * u + 1]);
    __syncthreads();
    // joined over the warps, into the first warp's place
    for (int i = threadIdx.x; i < rows * p.d; i += kFewThreads) {
        const int r = i / p.d, col = i - r * p.d;
        float mx = ms[0][r];
#pragma unroll
        for (int w = 1; w < kFewWarps; ++w) mx = fmaxf(mx, ms[w][r]);
        const float ref = mx == -INFINITY ? 0.0f : mx;
        float sum = 0.0f, total = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            const float f = ex2(ms[w][r] - ref);
            sum = fmaf(os[(w * kFewRows + r) * pitch + col], f, sum);
            total = fmaf(ls[w][r], f, total);
        }
        os[r * pitch + col] = sum;
        if (col == 0) {
            bm[r] = mx;
            bl[r] = total;
        }
    }
    if (ranks > 1) cluster_sync_all();
    else __syncthreads();
    // joined over the blocks: each finishes a part of the rows' pieces of eight columns
    const int pieces = p.d >> 3, total_pieces = rows * pieces, share = (total_pieces + ranks - 1) / ranks;
    for (int i = rank * share + threadIdx.x; i < min((rank + 1) * share, total_pieces); i += kFewThreads) {
        const int r = i / pieces, col = (i - r * pieces) * 8;
        float mr[kFewMaxCluster], mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < kFewMaxCluster; ++k) {
            mr[k] = -INFINITY;
            if (k < ranks) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(mr[k]) : "r"(mapa_shared(smem_u32(&bm[r]), (uint32_t)k)));
            mx = fmaxf(mx, mr[k]);
        }
        const float ref = mx == -INFINITY ? 0.0f : mx;
        float v[8] = {}, total = 0.0f;
        for (int k = 0; k < ranks; ++k) {
            float lk;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(lk) : "r"(mapa_shared(smem_u32(&bl[r]), (uint32_t)k)));
            float mk;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(mk) : "r"(mapa_shared(smem_u32(&bm[r]), (uint32_t)k)));
            const float f = ex2(mk - ref);
            total = fmaf(lk, f, total);
            const uint32_t at = mapa_shared(smem_u32(os + r * pitch + col), (uint32_t)k);
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                float x[4];
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(at + e * 4));
#pragma unroll
                for (int u = 0; u < 4; ++u) v[e + u] = fmaf(x[u], f, v[e + u]);
            }
        }
        const int h = r / p.Lq, lq = r - h * p.Lq, head = hk * p.group + h;
        const float inv = keys > 0 ? 1.0f / total : 0.0f;
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = keys > 0 ? pack_bf16(v[2 * u] * inv, v[2 * u + 1] * inv) : 0u;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out.data) + (int64_t)b * p.out.batch_stride +
                                  (int64_t)lq * p.out.token_stride + (int64_t)head * p.out.head_stride + col) =
            make_uint4(w[0], w[1], w[2], w[3]);
        if (p.lse && col == 0)
            p.lse[((int64_t)b * p.H + head) * p.Lq + lq] = keys > 0 ? (mx + log2f(total)) * kLn2 : -INFINITY;
    }
    if (ranks > 1) cluster_sync_all();              // the others may still read this block's results
}

template <int DS>
cudaError_t launch_few_kernel(const CUtensorMap& mk, const CUtensorMap& mv, const FewParams& p, int pairs, int ranks, cudaStream_t stream) {
    constexpr int kFewWarps = kWarpsOf<DS>, kFewThreads = 32 * kFewWarps;
    int smem = kFewWarps * kFewStages * 2 * p.chunks * kSliceChunk;
    const int join = kFewWarps * kFewRows * (DS * 16 + 8) * 4;
    if (smem < join) smem = join;
    smem += 1024;
    cudaError_t e = cudaFuncSetAttribute(xattn_few_kernel<DS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)pairs, (unsigned)ranks);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1;
    attr.val.clusterDim.y = (unsigned)ranks;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = ranks > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, xattn_few_kernel<DS>, mk, mv, p);
    if (e == cudaSuccess) count_launch(1);
    return e;
}

cudaError_t launch_forward_few(const CrossAttnArgs& a, int num_sms, cudaStream_t stream) {
    FewParams p{};
    CUtensorMap mk{}, mv{};
    if (a.Lk > 0 && (!make_heads_map(&mk, a.k, a.B, a.Lk, a.Hkv, a.d, kSlice, &p.ak) ||
                     !make_heads_map(&mv, a.v, a.B, a.Lk, a.Hkv, a.d, kSlice, &p.av)))
        return cudaErrorInvalidValue;
    p.q = a.q;
    p.out = a.out;
    p.lse = a.lse;
    p.kv_lens = a.kv_lens;
    p.c = a.scale * kLog2e;
    p.H = a.H;
    p.Hkv = a.Hkv;
    p.Lq = a.Lq;
    p.Lk = a.Lk;
    p.d = a.d;
    p.group = a.H / a.Hkv;
    p.chunks = (a.d + 63) / 64;
    p.dev_status = a.dev_status;
    // Blocks along the keys: the number that ends first, counted in slices of a warp; a block's start and join cost
    // about four.  One block fits an SM.
    const int pairs = a.B * a.Hkv;
    const int warps = p.chunks == 1 ? kWarpsOf<4> : kWarpsOf<8>;
    const int64_t slots = num_sms, slices = (a.Lk + kSlice - 1) / kSlice;
    int ranks = 1;
    int64_t best = 0;
    for (int r = 1; r <= kFewMaxCluster; r *= 2) {
        const int64_t cost = ((int64_t)pairs * r + slots - 1) / slots * ((slices + r * warps - 1) / (r * warps) + 4);
        if (best == 0 || cost < best) {
            best = cost;
            ranks = r;
        }
    }
    return p.chunks == 1 ? launch_few_kernel<4>(mk, mv, p, pairs, ranks, stream) : launch_few_kernel<8>(mk, mv, p, pairs, ranks, stream);
}

}  // namespace xattn
}  // namespace nvfp4
