// xattn_bwd.cu -- gradients of attention to an encoder's states of another
// length (nvfp4_cross_attention_backward).
//
//   P = 2^(c S - lse log2(e)), D_i = sum_c dO_ic O_ic, dS = P (dO V^T - D)
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO
// Three kernels: D (one pass over dO and O), dQ by query tiles, dK and dV by
// key tiles.  S and dO V^T are computed in both of the latter, seven tile
// products in place of five: the sums of either stay in tensor memory, so
// nothing is added in global memory and the order of every sum is fixed.
//
// dQ (dq_kernel): persistent, a work item is a 128-query tile of one head, its
// steps are key tiles of 128.  TMEM: two S, one dP = dO V^T, dQ.  dS overwrites
// its S as packed bf16, the A operand of dS K.  Once dS of a step is there, the
// issuing warp starts dP of the next step, dS K of this one and S of the one
// after next: the exponentials of the next step run meanwhile on an S that is
// there already.  The order runs on across work items; dQ of an item is read
// out between the next item's exponentials and its dS.
// dK, dV (dkv_kernel): a block has one key tile and a range of the query tiles
// of the heads that share it.  S and dP are computed transposed, so that P^T and
// dS^T are A operands in tensor memory (over S^T and dP^T, as packed bf16).
// dV += P^T dO and the next S^T run while the warps form dS^T; dK += dS^T Q and
// the next dP^T run under the next exponentials.
// In both, eight warps work on a tile: two per quarter of its rows, 64 columns
// each, whose packed result goes to the first 32 of their own columns.
#include "xattn.cuh"

namespace nvfp4 {
namespace xattn {

constexpr int kBwdThreads = 384;
constexpr int kBwdRegsLow = 64;               // 128 x 64 + 256 x 208 <= 384 x 168
constexpr int kBwdRegsHigh = 208;
static_assert(128 * kBwdRegsLow + 256 * kBwdRegsHigh <= kBwdThreads * 168, "register split exceeds the launch budget");

// A ring of shared-memory tiles; `count` loads so far.
struct TileRing {
    int n, slot;
    uint32_t phase;
    int count;
    __device__ explicit TileRing(int n_) : n(n_), slot(0), phase(0), count(0) {}
    __device__ void next() {
        ++count;
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
    // Waits (each with a limit) for the last load of every slot.
    __device__ void drain(uint64_t* full, const WaitCtx& w) {
        for (int i = 0; i < n && i < count; ++i) {
            if (--slot < 0) {
                slot = n - 1;
                phase ^= 1u;
            }
            mbar_wait_limit(&full[slot], phase, w, 1000000);
        }
    }
};

// A operand in TMEM, step kk: packed values of columns [0, 64) at `base`, of [64, 128) 64 columns on.
__device__ __forceinline__ uint32_t packed_a(uint32_t base, int kk) { return base + (kk >> 2) * 64 + (kk & 3) * 8; }

// ------------------------------------------------------------------ D
constexpr int kDeltaThreads = 256;
constexpr int kDeltaRows = 4;                 // rows of 16 lanes, each at once

__global__ void __launch_bounds__(kDeltaThreads) delta_kernel(const nvfp4_heads grad_out, const nvfp4_heads out, float* delta,
                                                              int64_t rows, int Lq, int H, int d) {
    const int lane = threadIdx.x & 15;
    const int64_t first = ((int64_t)blockIdx.x * kDeltaThreads + threadIdx.x) / 16 * kDeltaRows;
    uint4 a[kDeltaRows], b[kDeltaRows];
    int64_t at[kDeltaRows];
#pragma unroll
    for (int i = 0; i < kDeltaRows; ++i) {
        const int64_t r = first + i;                 // (b, l, h), heads innermost
        a[i] = b[i] = make_uint4(0, 0, 0, 0);
        at[i] = -1;
        if (r >= rows) continue;
        const int64_t bl = r / H, h = r - bl * H, bb = bl / Lq, l = bl - bb * Lq;
        at[i] = (bb * H + h) * Lq + l;
        if (lane * 8 < d) {
            a[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(grad_out.data) + bb * grad_out.batch_stride +
                                                        l * grad_out.token_stride + h * grad_out.head_stride + lane * 8));
            b[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(out.data) + bb * out.batch_stride +
                                                        l * out.token_stride + h * out.head_stride + lane * 8));
        }
    }
#pragma unroll
    for (int i = 0; i < kDeltaRows; ++i) {
        const uint32_t* x = reinterpret_cast<const uint32_t*>(&a[i]);
        const uint32_t* y = reinterpret_cast<const uint32_t*>(&b[i]);
        float s = 0.0f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            s = fmaf(__uint_as_float(x[u] << 16), __uint_as_float(y[u] << 16), s);
            s = fmaf(__uint_as_float(x[u] & 0xFFFF0000u), __uint_as_float(y[u] & 0xFFFF0000u), s);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0 && at[i] >= 0) delta[at[i]] = s;
    }
}

// ------------------------------------------------------------------ dQ
struct DqParams {
    MapAxes aq, ag, ak, av;
    nvfp4_heads dq;
    const float* lse;
    const float* delta;
    const int32_t* kv_lens;
    float c, scale;                           // scale * log2(e), scale
    int H, Hkv, Lq, Lk, d;
    int group, qtiles, items;
    int chunks, qbufs, kbufs, vbufs;
    int* dev_status;
};

struct DqItem {
    int b, h, q0, keys, steps;
};

__device__ __forceinline__ DqItem dq_item(const DqParams& p, int it) {
    DqItem r;
    const int bh = it / p.qtiles;
    r.q0 = (it - bh * p.qtiles) * kRows;
    r.b = bh / p.H;
    r.h = bh - r.b * p.H;
    r.keys = keys_of(p.kv_lens, r.b, p.Lk);
    r.steps = (r.keys + kRows - 1) / kRows;
    return r;
}

__device__ __forceinline__ int dq_next(const DqParams& p, int it, DqItem& item) {
    for (; it < p.items; it += gridDim.x) {
        item = dq_item(p, it);
        if (item.steps > 0) break;
    }
    return it;
}

// A walk over the steps of this block's items, in order.
struct DqWalk {
    int it, j;
    DqItem item;
    __device__ void start(const DqParams& p) {
        j = 0;
        it = dq_next(p, blockIdx.x, item);
    }
    __device__ bool valid(const DqParams& p) const { return it < p.items; }
    __device__ int keys_here() const { return min(item.keys - j * kRows, kRows); }
    __device__ bool last() const { return j == item.steps - 1; }
    __device__ void next(const DqParams& p) {
        if (++j == item.steps) {
            j = 0;
            it = dq_next(p, it + gridDim.x, item);
        }
    }
};

constexpr int kMaxQ = 4, kMaxK = 4, kMaxV = 4;
constexpr uint32_t kDqS = 0, kDqP = 256, kDqO = 384;      // S: [128 (s & 1), + 128); dP; dQ

__global__ void __launch_bounds__(kBwdThreads, 1)
xattn_dq_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_g,
                const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v, const DqParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t q_full[kMaxQ], q_empty[kMaxQ], k_full[kMaxK], k_empty[kMaxK], v_full[kMaxV], v_empty[kMaxV];
    __shared__ __align__(8) uint64_t s_full[2], dp_full, ds_ready, dq_full, drain;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tile_bytes = p.chunks * kChunk;
    uint8_t* k_tiles = smem + p.qbufs * tile_bytes;
    uint8_t* v_tiles = k_tiles + p.kbufs * tile_bytes;
    WaitCtx wc{&abort_sh, p.dev_status};

    if (threadIdx.x == 0) {
        abort_sh = 0;
        for (int i = 0; i < kMaxQ; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < kMaxK; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < kMaxV; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        mbar_init(&dp_full, 1);
        mbar_init(&ds_ready, 8);                    // the eight warps
        mbar_init(&dq_full, 1);
        mbar_init(&drain, 1);
        fence_barrier_init();
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_g);
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base_sh, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;

    if (warp < 4) {
        regs_dec<kBwdRegsLow>();
        if (warp == 0) {
            // -------------------------------------------------------- loads: Q, K, dO, V of an item, then K and V of its steps
            TileRing rq(p.qbufs), rk(p.kbufs), rv(p.vbufs);
            DqWalk w;
            bool ok = true;
            auto load = [&](TileRing& ring, uint64_t* full, uint64_t* empty, uint8_t* tiles, const CUtensorMap* map, int h, int l,
                            int b) {
                if (!warp_wait(&empty[ring.slot], ring.phase ^ 1u, wc)) return false;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&full[ring.slot], (uint32_t)tile_bytes);
                    load_tile(tiles + ring.slot * tile_bytes, map, &full[ring.slot], p.chunks, kChunk, h, l, b);
                }
                __syncwarp();
                ring.next();
                return true;
            };
            for (w.start(p); ok && w.valid(p); w.next(p)) {
                const DqItem& i = w.item;
                const int hk = i.h / p.group;
                ok = (w.j > 0 || load(rq, q_full, q_empty, smem, &tmap_q, i.h * p.aq.h, i.q0, i.b * p.aq.b)) &&
                     load(rk, k_full, k_empty, k_tiles, &tmap_k, hk * p.ak.h, w.j * kRows, i.b * p.ak.b) &&
                     (w.j > 0 || load(rq, q_full, q_empty, smem, &tmap_g, i.h * p.ag.h, i.q0, i.b * p.ag.b)) &&
                     load(rv, v_full, v_empty, v_tiles, &tmap_v, hk * p.av.h, w.j * kRows, i.b * p.av.b);
            }
            if (!ok && lane == 0) {                 // a block that gave up still waits for its loads in flight
                int dummy = 0;
                WaitCtx w2{&dummy, p.dev_status};
                rq.drain(q_full, w2);
                rk.drain(k_full, w2);
                rv.drain(v_full, w2);
            }
            __syncwarp();
        } else if (warp == 1) {
            // -------------------------------------------------------- products
            const uint32_t q_sm = smem_u32(smem), k_sm = smem_u32(k_tiles), v_sm = smem_u32(v_tiles);
            const int dsteps = (p.d + 15) >> 4;
            const uint32_t idesc_o = idesc_kmn(dsteps * 16);
            TileRing ks(p.kbufs), kq(p.kbufs), rv(p.vbufs);      // K as S and as dQ use it, V
            TileRing qs(p.qbufs), qp(p.qbufs);                   // Q tiles (even entries), dO tiles (odd ones)
            qp.next();
            DqWalk ws, wp, wq;                                   // steps of S, dP, dQ
            ws.start(p);
            wp = wq = ws;
            uint32_t s_at = 0;                                   // S products so far
            uint32_t done = 0;                                   // dS so far
            int q_slot = 0, g_slot = 0;
            bool ok = true;

            auto issue_s = [&]() {
                if (ws.j == 0) {
                    q_slot = qs.slot;
                    if (!warp_wait(&q_full[qs.slot], qs.phase, wc)) return false;
                    qs.next();
                    qs.next();
                }
                if (!warp_wait(&k_full[ks.slot], ks.phase, wc)) return false;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t qt = q_sm + q_slot * tile_bytes, kt = k_sm + ks.slot * tile_bytes;
                    const uint32_t idesc = idesc_kk((ws.keys_here() + 15) & ~15);
                    for (int kk = 0; kk < dsteps; ++kk)
                        tc_mma_bf16(tmem + kDqS + (s_at & 1u) * 128, desc_kmajor(qt, kk, kChunk), desc_kmajor(kt, kk, kChunk),
                                    idesc, kk != 0 ? 1u : 0u);
                    tc_commit(&s_full[s_at & 1u]);
                    if (ws.last()) tc_commit(&q_empty[q_slot]);
                }
                __syncwarp();
                ks.next();
                ++s_at;
                ws.next(p);
                return true;
            };
            auto issue_dp = [&]() {
                if (wp.j == 0) {
                    g_slot = qp.slot;
                    if (!warp_wait(&q_full[qp.slot], qp.phase, wc)) return false;
                    qp.next();
                    qp.next();
                }
                if (!warp_wait(&v_full[rv.slot], rv.phase, wc)) return false;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t gt = q_sm + g_slot * tile_bytes, vt = v_sm + rv.slot * tile_bytes;
                    const uint32_t idesc = idesc_kk((wp.keys_here() + 15) & ~15);
                    for (int kk = 0; kk < dsteps; ++kk)
                        tc_mma_bf16(tmem + kDqP, desc_kmajor(gt, kk, kChunk), desc_kmajor(vt, kk, kChunk), idesc,
                                    kk != 0 ? 1u : 0u);
                    tc_commit(&dp_full);
                    tc_commit(&v_empty[rv.slot]);
                    if (wp.last()) tc_commit(&q_empty[g_slot]);
                }
                __syncwarp();
                rv.next();
                wp.next(p);
                return true;
            };

            if (ws.valid(p)) {
                ok = issue_s() && issue_dp();
                if (ok && ws.valid(p)) ok = issue_s();
            }
            while (ok && wq.valid(p)) {
                const int n = wq.keys_here();
                ok = warp_wait(&ds_ready, done & 1u, wc);
                if (!ok) break;
                if (wp.valid(p) && !(ok = issue_dp())) break;
                if ((n & 15) != 0 && wq.item.keys < p.Lk) {
                    // keys past the sample's length meet dS = 0, but may be NaN: the rest of the last
                    // 16 rows reads as zeros (rows past the tensor already do; S of the step is done)
                    uint8_t* row = k_tiles + kq.slot * tile_bytes;
                    const int rows = 16 - (n & 15);
                    for (int i = lane; i < rows * 8 * p.chunks; i += 32) {
                        const int c = i / (rows * 8), r = i - c * rows * 8;
                        *reinterpret_cast<uint4*>(row + c * kChunk + n * 128 + r * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t kt = k_sm + kq.slot * tile_bytes, a = tmem + kDqS + (done & 1u) * 128;
                    const int ksteps = (n + 15) >> 4;
                    for (int kk = 0; kk < ksteps; ++kk)
                        tc_mma_bf16_ta(tmem + kDqO, packed_a(a, kk), desc_mnmajor(kt, kk, kChunk), idesc_o,
                                       (wq.j | kk) != 0 ? 1u : 0u);
                    tc_commit(&k_empty[kq.slot]);
                    if (wq.last()) tc_commit(&dq_full);
                }
                __syncwarp();
                kq.next();
                ++done;
                wq.next(p);
                if (ws.valid(p)) ok = issue_s();
            }
            if (elect_one()) tc_commit(&drain);
            __syncwarp();
            int dummy = 0;
            WaitCtx w2{&dummy, p.dev_status};
            mbar_wait(&drain, 0, w2);
        }
    } else {
        regs_inc<kBwdRegsHigh>();
        // ------------------------------------------------------------ dS, and dQ of finished items
        const int g = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint32_t tbase = tmem + lane_base + g * 64;
        uint32_t step = 0, outs = 0;
        bool ok = true;

        auto row_at = [&](const DqItem& i) {
            return static_cast<uint16_t*>(p.dq.data) + (int64_t)i.b * p.dq.batch_stride + (int64_t)(i.q0 + r) * p.dq.token_stride +
                   (int64_t)i.h * p.dq.head_stride;
        };
        auto read_out = [&](const DqItem& i) {
            if (!warp_wait(&dq_full, outs & 1u, wc)) return false;
            ++outs;
            tc_fence_after();
            uint16_t* dst = row_at(i);
#pragma unroll
            for (int c2 = 0; c2 < 2; ++c2) {
                const int col = g * 64 + c2 * 32;
                if (col >= p.d) break;
                uint32_t o[32];
                tmem_ld_32x32b_x32(tbase + kDqO + c2 * 32, o);
                tmem_ld_wait();
                if (i.q0 + r < p.Lq) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        if (col + e >= p.d) break;
                        uint32_t w[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            w[u] = pack_bf16(__uint_as_float(o[e + 2 * u]) * p.scale, __uint_as_float(o[e + 2 * u + 1]) * p.scale);
                        *reinterpret_cast<uint4*>(dst + col + e) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            return true;
        };

        DqItem prev;
        bool pending = false;
        for (int it = blockIdx.x; ok && it < p.items; it += gridDim.x) {
            const DqItem item = dq_item(p, it);
            const bool have = item.q0 + r < p.Lq;
            if (item.steps == 0) {
                if (have)
                    for (int i = g * 64; i < min(p.d, g * 64 + 64); i += 8)
                        *reinterpret_cast<uint4*>(row_at(item) + i) = make_uint4(0, 0, 0, 0);
                continue;
            }
            const int64_t at = ((int64_t)item.b * p.H + item.h) * p.Lq + item.q0 + r;
            const float lse2 = have ? __ldg(p.lse + at) * kLog2e : INFINITY, dl = have ? __ldg(p.delta + at) : 0.0f;
            for (int j = 0; j < item.steps; ++j, ++step) {
                const int n = min(max(item.keys - j * kRows - g * 64, 0), 64);      // this warp's keys
                const uint32_t ts = tbase + kDqS + (step & 1u) * 128, tp = tbase + kDqP;
                if (!(ok = warp_wait(&s_full[step & 1u], (step >> 1) & 1u, wc))) break;
                tc_fence_after();
                uint32_t v[64];
#pragma unroll
                for (int c2 = 0; c2 < 2; ++c2)
                    if (c2 * 32 < n) tmem_ld_32x32b_x32(ts + c2 * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[c2 * 32]));
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 64; ++i) v[i] = __float_as_uint(ex2(fmaf(__uint_as_float(v[i]), p.c, -lse2)));
                if (pending) {
                    if (!(ok = read_out(prev))) break;
                    pending = false;
                }
                if (!(ok = warp_wait(&dp_full, step & 1u, wc))) break;
                tc_fence_after();
                uint32_t w[32];
#pragma unroll
                for (int c2 = 0; c2 < 2; ++c2) {
                    if (c2 * 32 >= n) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[c2 * 16 + i] = 0;
                        continue;
                    }
                    uint32_t dp[32];
                    tmem_ld_32x32b_x32(tp + c2 * 32, dp);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        dp[i] = __float_as_uint((__uint_as_float(dp[i]) - dl) * __uint_as_float(v[c2 * 32 + i]));
                    if (n < 64) {
                        // keys past the length: zero, whatever was computed there
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c2 * 32 + i >= n) dp[i] = 0;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        w[c2 * 16 + i] = pack_bf16(__uint_as_float(dp[2 * i]), __uint_as_float(dp[2 * i + 1]));
                }
                if (n > 0) tmem_st_x32(ts, w);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ds_ready);
            }
            prev = item;
            pending = ok;
        }
        if (ok && pending) read_out(prev);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ dK, dV
struct DkvParams {
    MapAxes aq, ag, ak, av;
    nvfp4_heads dk, dv;
    const float* lse;
    const float* delta;
    const int32_t* kv_lens;
    float* partial;                           // [chunk][unit][dk, dv][d / 4][128][4]; null: one chunk, written out directly
    float c, scale;
    int H, Hkv, Lq, Lk, d;
    int group, qtiles, ktiles, steps, splits; // query tiles of a key tile (all heads that share it), ranges of them
    int chunks, qbufs;
    int* dev_status;
};

constexpr int kMaxQG = 8;
constexpr uint32_t kKvS = 0, kKvP = 128, kKvV = 256, kKvK = 384;

__global__ void __launch_bounds__(kBwdThreads, 1)
xattn_dkv_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_g,
                 const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v, const DkvParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t qg_full[kMaxQG], qg_empty[kMaxQG], k_full, v_full;
    __shared__ __align__(8) uint64_t s_full, dp_full, p_ready, ds_ready, st_full[2], st_empty[2], drain;
    __shared__ __align__(16) float st_lse[2][kRows], st_delta[2][kRows];
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;

    const int unit = blockIdx.x / p.splits, split = blockIdx.x - unit * p.splits;
    const int bh = unit / p.ktiles, k0 = (unit - bh * p.ktiles) * kRows;
    const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
    const int keys = keys_of(p.kv_lens, b, p.Lk);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (k0 >= keys) {
        // no valid key: zeros where no later kernel writes them
        if (!p.partial)
            for (int i = threadIdx.x; i < min(kRows, p.Lk - k0) * (p.d / 8); i += kBwdThreads) {
                const int row = i / (p.d / 8), col = (i - row * (p.d / 8)) * 8;
                for (const nvfp4_heads* t : {&p.dk, &p.dv})
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(t->data) + (int64_t)b * t->batch_stride +
                                              (int64_t)(k0 + row) * t->token_stride + (int64_t)hk * t->head_stride + col) =
                        make_uint4(0, 0, 0, 0);
            }
        return;
    }
    const int first = (int)((int64_t)p.steps * split / p.splits), last = (int)((int64_t)p.steps * (split + 1) / p.splits);

    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tile_bytes = p.chunks * kChunk;
    uint8_t* qg_tiles = smem + 2 * tile_bytes;
    WaitCtx wc{&abort_sh, p.dev_status};

    if (threadIdx.x == 0) {
        abort_sh = 0;
        for (int i = 0; i < kMaxQG; ++i) {
            mbar_init(&qg_full[i], 1);
            mbar_init(&qg_empty[i], 1);
        }
        mbar_init(&k_full, 1);
        mbar_init(&v_full, 1);
        mbar_init(&s_full, 1);
        mbar_init(&dp_full, 1);
        mbar_init(&p_ready, 8);                     // the eight warps
        mbar_init(&ds_ready, 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&st_full[i], 32);
            mbar_init(&st_empty[i], 8);
        }
        mbar_init(&drain, 1);
        fence_barrier_init();
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_g);
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base_sh, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;

    // head and first query of step t
    auto place = [&](int t, int& h, int& q0) {
        const int in_group = t / p.qtiles;
        h = hk * p.group + in_group;
        q0 = (t - in_group * p.qtiles) * kRows;
    };

    if (warp < 4) {
        regs_dec<kBwdRegsLow>();
        if (warp == 0) {
            // -------------------------------------------------------- loads: K, then Q and dO of the steps (V after the first Q)
            TileRing ring(p.qbufs);
            bool ok = true;
            auto load = [&](const CUtensorMap* map, int h, int q0, int bb) {
                if (!warp_wait(&qg_empty[ring.slot], ring.phase ^ 1u, wc)) return false;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&qg_full[ring.slot], (uint32_t)tile_bytes);
                    load_tile(qg_tiles + ring.slot * tile_bytes, map, &qg_full[ring.slot], p.chunks, kChunk, h, q0, bb);
                }
                __syncwarp();
                ring.next();
                return true;
            };
            if (elect_one()) {
                mbar_arrive_expect_tx(&k_full, (uint32_t)tile_bytes);
                load_tile(smem, &tmap_k, &k_full, p.chunks, kChunk, hk * p.ak.h, k0, b * p.ak.b);
                mbar_arrive_expect_tx(&v_full, (uint32_t)tile_bytes);
                load_tile(smem + tile_bytes, &tmap_v, &v_full, p.chunks, kChunk, hk * p.av.h, k0, b * p.av.b);
            }
            __syncwarp();
            for (int t = first; ok && t < last; ++t) {
                int h, q0;
                place(t, h, q0);
                ok = load(&tmap_q, h * p.aq.h, q0, b * p.aq.b) && load(&tmap_g, h * p.ag.h, q0, b * p.ag.b);
            }
            if (!ok && lane == 0) {                 // a block that gave up still waits for its loads in flight
                int dummy = 0;
                WaitCtx w2{&dummy, p.dev_status};
                mbar_wait_limit(&k_full, 0, w2, 1000000);
                mbar_wait_limit(&v_full, 0, w2, 1000000);
                ring.drain(qg_full, w2);
            }
            __syncwarp();
        } else if (warp == 1) {
            // -------------------------------------------------------- products
            const uint32_t k_sm = smem_u32(smem), v_sm = k_sm + tile_bytes, qg_sm = v_sm + tile_bytes;
            const int dsteps = (p.d + 15) >> 4;
            const uint32_t idesc_o = idesc_kmn(dsteps * 16);
            TileRing rs(p.qbufs), rp(p.qbufs), rv(p.qbufs), rk(p.qbufs);    // Q for S, dO for dP, dO for dV, Q for dK
            rp.next();
            rv.next();
            auto queries = [&](int t) { return min(p.Lq - (t % p.qtiles) * kRows, kRows); };
            // S^T or dP^T of step t: rows = keys, columns = queries
            auto scores = [&](int t, TileRing& ring, uint32_t a_sm, uint32_t col, uint64_t* bar) {
                if (!warp_wait(&qg_full[ring.slot], ring.phase, wc)) return false;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t bt = qg_sm + ring.slot * tile_bytes;
                    const uint32_t idesc = idesc_kk((queries(t) + 15) & ~15);
                    for (int kk = 0; kk < dsteps; ++kk)
                        tc_mma_bf16(tmem + col, desc_kmajor(a_sm, kk, kChunk), desc_kmajor(bt, kk, kChunk), idesc,
                                    kk != 0 ? 1u : 0u);
                    tc_commit(bar);
                }
                __syncwarp();
                ring.next();
                ring.next();
                return true;
            };
            // dV or dK += (P^T or dS^T) (dO or Q)
            auto update = [&](int t, TileRing& ring, uint32_t a, uint32_t col) {
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t bt = qg_sm + ring.slot * tile_bytes;
                    const int ksteps = (queries(t) + 15) >> 4;
                    for (int kk = 0; kk < ksteps; ++kk)
                        tc_mma_bf16_ta(tmem + col, packed_a(tmem + a, kk), desc_mnmajor(bt, kk, kChunk), idesc_o,
                                       t > first || kk != 0 ? 1u : 0u);
                    tc_commit(&qg_empty[ring.slot]);
                }
                __syncwarp();
                ring.next();
                ring.next();
            };
            bool ok = warp_wait(&k_full, 0, wc) && scores(first, rs, k_sm, kKvS, &s_full) && warp_wait(&v_full, 0, wc) &&
                      scores(first, rp, v_sm, kKvP, &dp_full);
            for (int t = first; ok && t < last; ++t) {
                const uint32_t ph = (uint32_t)(t - first) & 1u;
                if (!(ok = warp_wait(&p_ready, ph, wc))) break;
                update(t, rv, kKvS, kKvV);
                if (t + 1 < last && !(ok = scores(t + 1, rs, k_sm, kKvS, &s_full))) break;
                if (!(ok = warp_wait(&ds_ready, ph, wc))) break;
                update(t, rk, kKvP, kKvK);
                if (t + 1 < last) ok = scores(t + 1, rp, v_sm, kKvP, &dp_full);
            }
            if (elect_one()) tc_commit(&drain);
            __syncwarp();
            int dummy = 0;
            WaitCtx w2{&dummy, p.dev_status};
            mbar_wait(&drain, 0, w2);
        } else if (warp == 2) {
            // -------------------------------------------------------- lse (times log2(e)) and D of the steps' queries
            bool ok = true;
            for (int t = first; ok && t < last; ++t) {
                const int s = (t - first) & 1;
                int h, q0;
                place(t, h, q0);
                const int64_t at = ((int64_t)b * p.H + h) * p.Lq + q0;
                float l[4], dl[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool have = q0 + lane + 32 * i < p.Lq;
                    l[i] = have ? __ldg(p.lse + at + lane + 32 * i) * kLog2e : INFINITY;
                    dl[i] = have ? __ldg(p.delta + at + lane + 32 * i) : 0.0f;
                }
                if (!(ok = warp_wait(&st_empty[s], (((uint32_t)(t - first) >> 1) & 1u) ^ 1u, wc))) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    st_lse[s][lane + 32 * i] = l[i];
                    st_delta[s][lane + 32 * i] = dl[i];
                }
                mbar_arrive(&st_full[s]);
            }
        }
    } else {
        regs_inc<kBwdRegsHigh>();
        // ------------------------------------------------------------ P^T and dS^T, a key per thread
        const int g = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint32_t ts = tmem + lane_base + kKvS + g * 64, tp = tmem + lane_base + kKvP + g * 64;
        bool ok = true;
        for (int t = first; t < last; ++t) {
            const int s = (t - first) & 1;
            const uint32_t ph = (uint32_t)(t - first) & 1u;
            const float4* lse4 = reinterpret_cast<const float4*>(&st_lse[s][g * 64]);
            const float4* del4 = reinterpret_cast<const float4*>(&st_delta[s][g * 64]);
            if (!(ok = warp_wait(&st_full[s], ((uint32_t)(t - first) >> 1) & 1u, wc) && warp_wait(&s_full, ph, wc))) break;
            tc_fence_after();
            uint32_t v[64], w[16];
            tmem_ld_32x32b_x32(ts, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
            tmem_ld_32x32b_x32(ts + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
            tmem_ld_wait();
            // columns past the last query hold anything: -lse = -infinity alone would leave NaN there
            const int nq = p.Lq - (t % p.qtiles) * kRows - g * 64;
            if (nq < 64) {
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    if (i >= nq) v[i] = 0;
            }
#pragma unroll
            for (int c2 = 0; c2 < 2; ++c2) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 l = lse4[c2 * 8 + i];
                    uint32_t* e = v + c2 * 32 + 4 * i;
                    e[0] = __float_as_uint(ex2(fmaf(__uint_as_float(e[0]), p.c, -l.x)));
                    e[1] = __float_as_uint(ex2(fmaf(__uint_as_float(e[1]), p.c, -l.y)));
                    e[2] = __float_as_uint(ex2(fmaf(__uint_as_float(e[2]), p.c, -l.z)));
                    e[3] = __float_as_uint(ex2(fmaf(__uint_as_float(e[3]), p.c, -l.w)));
                    w[2 * i] = pack_bf16(__uint_as_float(e[0]), __uint_as_float(e[1]));
                    w[2 * i + 1] = pack_bf16(__uint_as_float(e[2]), __uint_as_float(e[3]));
                }
                tmem_st_x16(ts + c2 * 16, w);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready);

            if (!(ok = warp_wait(&dp_full, ph, wc))) break;
            tc_fence_after();
#pragma unroll
            for (int c2 = 0; c2 < 2; ++c2) {
                uint32_t dp[32];
                tmem_ld_32x32b_x32(tp + c2 * 32, dp);
                tmem_ld_wait();
                if (nq < 64) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c2 * 32 + i >= nq) dp[i] = 0;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 dl = del4[c2 * 8 + i];
                    const int at = c2 * 32 + 4 * i;
                    const float a0 = (__uint_as_float(dp[4 * i]) - dl.x) * __uint_as_float(v[at]);
                    const float a1 = (__uint_as_float(dp[4 * i + 1]) - dl.y) * __uint_as_float(v[at + 1]);
                    const float a2 = (__uint_as_float(dp[4 * i + 2]) - dl.z) * __uint_as_float(v[at + 2]);
                    const float a3 = (__uint_as_float(dp[4 * i + 3]) - dl.w) * __uint_as_float(v[at + 3]);
                    w[2 * i] = pack_bf16(a0, a1);
                    w[2 * i + 1] = pack_bf16(a2, a3);
                }
                // over this warp's own columns, which it has read so far
                tmem_st_x16(tp + c2 * 16, w);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&st_empty[s]);
                mbar_arrive(&ds_ready);
            }
        }
        // the sums: this thread's key, 64 of the d columns
        if (ok && warp_wait(&drain, 0, wc)) {
            tc_fence_after();
#pragma unroll 1
            for (int o = 0; o < 2; ++o) {
                const float f = o == 0 ? p.scale : 1.0f;
                const nvfp4_heads& t = o == 0 ? p.dk : p.dv;
                const uint32_t from = tmem + lane_base + (o == 0 ? kKvK : kKvV) + g * 64;
                uint16_t* dst = static_cast<uint16_t*>(t.data) + (int64_t)b * t.batch_stride + (int64_t)(k0 + r) * t.token_stride +
                                (int64_t)hk * t.head_stride;
                float* part = p.partial + (((int64_t)split * (gridDim.x / p.splits) + unit) * 2 + o) * p.d * kRows;
#pragma unroll
                for (int c2 = 0; c2 < 2; ++c2) {
                    const int col = g * 64 + c2 * 32;
                    if (col >= p.d) break;
                    uint32_t x[32];
                    tmem_ld_32x32b_x32(from + c2 * 32, x);
                    tmem_ld_wait();
                    if (p.partial) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            if (col + e >= p.d) break;
                            *reinterpret_cast<uint4*>(part + ((int64_t)((col + e) >> 2) * kRows + r) * 4) =
                                make_uint4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                        }
                    } else if (k0 + r < p.Lk) {
                        const bool valid = k0 + r < keys;
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            if (col + e >= p.d) break;
                            uint32_t y[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                y[u] = valid ? pack_bf16(__uint_as_float(x[e + 2 * u]) * f, __uint_as_float(x[e + 2 * u + 1]) * f) : 0u;
                            *reinterpret_cast<uint4*>(dst + col + e) = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// dK and dV from the partial sums of `splits` ranges, in their order (splits = 0: zeros).
constexpr int kJoinThreads = 256;

__global__ void __launch_bounds__(kJoinThreads) join_kernel(const float* partial, int splits, int64_t units, nvfp4_heads dk,
                                                            nvfp4_heads dv, const int32_t* kv_lens, float scale, int Hkv, int Lk,
                                                            int ktiles, int d) {
    const int pieces = d / 8;                         // of eight columns
    const int r = threadIdx.x % kRows;
    int64_t rest = (int64_t)blockIdx.x * (kJoinThreads / kRows) + threadIdx.x / kRows;
    const int piece = (int)(rest % pieces);
    rest /= pieces;
    const int o = (int)(rest & 1);
    const int64_t unit = rest >> 1;
    if (unit >= units) return;
    const int64_t bh = unit / ktiles;
    const int b = (int)(bh / Hkv), hk = (int)(bh - (int64_t)b * Hkv), key = (int)(unit - bh * ktiles) * kRows + r;
    if (key >= Lk) return;
    float s[8] = {};
    if (key < keys_of(kv_lens, b, Lk)) {
        const float* src = partial + ((unit * 2 + o) * d + piece * 8) * kRows + r * 4;
#pragma unroll 4
        for (int c = 0; c < splits; ++c, src += units * 2 * d * kRows) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(src));
            const float4 y = __ldg(reinterpret_cast<const float4*>(src + 4 * kRows));
            s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w;
            s[4] += y.x, s[5] += y.y, s[6] += y.z, s[7] += y.w;
        }
        if (o == 0)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] *= scale;
    }
    const nvfp4_heads& t = o == 0 ? dk : dv;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(t.data) + (int64_t)b * t.batch_stride + (int64_t)key * t.token_stride +
                              (int64_t)hk * t.head_stride + piece * 8) =
        make_uint4(pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]), pack_bf16(s[4], s[5]), pack_bf16(s[6], s[7]));
}

// Ranges of the query tiles of a key tile: the number that ends first, counted in steps, where each block costs
// kSplitCost steps beside its own (start, last sums and their share of the join).
constexpr int kSplitCost = 3;
constexpr int kPlanSms = 148;

int split_count(int64_t units, int64_t steps) {
    if (units == 0 || steps == 0) return 0;
    int64_t best = 0, best_cost = 0;
    for (int64_t c = 1; c <= steps && c <= 64; ++c) {
        const int64_t cost = (units * c + kPlanSms - 1) / kPlanSms * ((steps + c - 1) / c + kSplitCost);
        if (best == 0 || cost < best_cost) {
            best = c;
            best_cost = cost;
        }
    }
    return (int)best;
}

struct BwdPlan {
    int64_t units, steps, delta_bytes, partial_bytes;
    int splits;
};

BwdPlan plan_backward(int64_t B, int64_t H, int64_t Hkv, int64_t Lq, int64_t Lk, int64_t d) {
    BwdPlan p;
    p.units = B * Hkv * ((Lk + kRows - 1) / kRows);
    p.steps = H / Hkv * ((Lq + kRows - 1) / kRows);
    p.splits = split_count(p.units, p.steps);
    p.delta_bytes = (B * H * Lq * 4 + 15) / 16 * 16;
    p.partial_bytes = p.splits > 1 ? p.splits * p.units * 2 * d * kRows * 4 : 0;
    return p;
}

cudaError_t prepare_kernel(const void* kernel, int smem) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

}  // namespace xattn

size_t cross_attention_backward_workspace(int64_t B, int64_t H, int64_t Hkv, int64_t Lq, int64_t Lk, int64_t d) {
    const xattn::BwdPlan p = xattn::plan_backward(B, H, Hkv, Lq, Lk, d);
    return (size_t)(p.delta_bytes + p.partial_bytes);
}

cudaError_t launch_cross_attention_backward(const CrossAttnArgs& a, int num_sms, cudaStream_t stream) {
    using namespace xattn;
    const BwdPlan plan = plan_backward(a.B, a.H, a.Hkv, a.Lq, a.Lk, a.d);
    float* delta = static_cast<float*>(a.workspace);
    float* partial = plan.splits > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + plan.delta_bytes) : nullptr;
    const int qtiles = (a.Lq + kRows - 1) / kRows, ktiles = (a.Lk + kRows - 1) / kRows;
    const int chunks = (a.d + 63) / 64, tile_bytes = chunks * kChunk;
    CUtensorMap mq{}, mg{}, mk{}, mv{};
    MapAxes aq{}, ag{}, ak{}, av{};
    if (a.Lq > 0 && a.Lk > 0 &&
        (!make_heads_map(&mq, a.q, a.B, a.Lq, a.H, a.d, kRows, &aq) || !make_heads_map(&mg, a.grad_out, a.B, a.Lq, a.H, a.d, kRows, &ag) ||
         !make_heads_map(&mk, a.k, a.B, a.Lk, a.Hkv, a.d, kRows, &ak) || !make_heads_map(&mv, a.v, a.B, a.Lk, a.Hkv, a.d, kRows, &av)))
        return cudaErrorInvalidValue;
    cudaError_t e;
    int launches = 0;
    if (a.Lq > 0) {
        const int64_t rows = (int64_t)a.B * a.Lq * a.H;
        const int64_t per = kDeltaThreads / 16 * kDeltaRows;
        delta_kernel<<<(unsigned)((rows + per - 1) / per), kDeltaThreads, 0, stream>>>(a.grad_out, a.out, delta, rows, a.Lq, a.H, a.d);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        DqParams p{aq, ag, ak, av, a.dq, a.lse, delta, a.kv_lens, a.scale * kLog2e, a.scale, a.H, a.Hkv, a.Lq, a.Lk, a.d,
                   a.H / a.Hkv, qtiles, a.B * a.H * qtiles, chunks, chunks == 1 ? 4 : 3, chunks == 1 ? 4 : 3, chunks == 1 ? 4 : 1,
                   a.dev_status};
        const int smem = (p.qbufs + p.kbufs + p.vbufs) * tile_bytes + 1024;
        if ((e = prepare_kernel(reinterpret_cast<const void*>(xattn_dq_kernel), smem)) != cudaSuccess) return e;
        xattn_dq_kernel<<<p.items < num_sms ? p.items : num_sms, kBwdThreads, smem, stream>>>(mq, mg, mk, mv, p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        launches += 2;
    }
    if (plan.units > 0 && plan.splits > 0) {
        DkvParams p{aq, ag, ak, av, a.dk, a.dv, a.lse, delta, a.kv_lens, partial, a.scale * kLog2e, a.scale, a.H, a.Hkv, a.Lq, a.Lk,
                    a.d, a.H / a.Hkv, qtiles, ktiles, (int)plan.steps, plan.splits, chunks, chunks == 1 ? 8 : 4, a.dev_status};
        const int smem = (2 + p.qbufs) * tile_bytes + 1024;
        if ((e = prepare_kernel(reinterpret_cast<const void*>(xattn_dkv_kernel), smem)) != cudaSuccess) return e;
        xattn_dkv_kernel<<<(unsigned)(plan.units * plan.splits), kBwdThreads, smem, stream>>>(mq, mg, mk, mv, p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        ++launches;
    }
    if (plan.units > 0 && plan.splits != 1) {
        const int64_t threads = plan.units * 2 * (a.d / 8) * kRows;
        join_kernel<<<(unsigned)((threads + kJoinThreads - 1) / kJoinThreads), kJoinThreads, 0, stream>>>(
            partial, plan.splits, plan.units, a.dk, a.dv, a.kv_lens, a.scale, a.Hkv, a.Lk, ktiles, a.d);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        ++launches;
    }
    count_launch(launches);
    return cudaSuccess;
}

}  // namespace nvfp4
