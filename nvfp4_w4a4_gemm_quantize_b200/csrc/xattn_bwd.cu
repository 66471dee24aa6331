// xattn_bwd.cu -- gradients of attention to an encoder's states of another
// length (nvfp4_cross_attention_backward).
//
//   P = 2^(c S - lse log2(e)), D_i = sum_c dO_ic O_ic, dS = P (dO V^T - D)
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO
// Three kernels: D (one pass over dO and O, where the states are more than one
// key tile), dQ by query tiles (apart for samples of more key tiles and of one,
// which forms its D itself), dK and dV by key tiles.  S and dO V^T are
// computed in both of the latter, seven tile products in place of five: the sums
// of either stay in tensor memory, so nothing is added in global memory and the
// order of every sum is fixed.
// P and dS are rounded to bf16 for their products, as K, Q and dO are bf16 and the
// tensor core wants both operands in one type: the gradients are 2.4e-3 off the
// formula in 64 bits (relative, in the norm) where FP32 arithmetic rounded once is
// 1.7e-3.  D of samples of several key tiles comes from the bf16 O, which it would
// otherwise take another pass over the keys to replace; its error counts where
// dP - D is small, with few keys, and those samples form D from P and dP.
// B200, 2 x 8192 queries x (512, 389) states, 24 heads of 128, each kernel alone: D
// 36 us (its bytes 31), dQ 167, dK and dV 195, their join 21; the whole 412 in a
// burst, 438 sustained under the 1000 W limit.  A step takes 2510 to 2580 cycles in
// dQ, 1536 of them the tensor core's, and 3150 to 3300 in dK and dV, 2048 of them
// (the slope over 512 to 2048 keys; starts and ends bring the whole launch to 43 and
// 58 % of the tensor core): the one issuing warp shares its scheduler with busy
// warps, and its waits on barriers that are complete take 170 to 290 cycles each.
// (Two issuing warps, one a pair of products, were slower, by a tenth for dK and dV:
// their products alternate on the tensor core.)
//
// dQ (dq_kernel): persistent, a work item is a 128-query tile of one head, its
// steps are key tiles of 128.  TMEM: two S, one dP = dO V^T, dQ.  dS overwrites
// its S as packed bf16, the A operand of dS K.  Once dS of a step is there, the
// issuing warp starts dP of the next step, dS K of this one and S of the one
// after next: the exponentials of the next step run meanwhile on an S that is
// there already.  The order runs on across work items; dQ of an item is read
// out between the next item's exponentials and its dS, and goes out by TMA from
// its own dO tile.
// dK, dV (dkv_kernel): a block has one key tile and a range of the query tiles
// of the heads that share it.  S and dP are computed transposed, so that P^T and
// dS^T are A operands in tensor memory (over S^T and dP^T, as packed bf16).
// dV += P^T dO and the next S^T run while the warps form dS^T; dK += dS^T Q and
// the next dP^T run under the next exponentials.
// In both, sixteen warps work on a tile: four per quarter of its rows, 32 columns
// each, whose packed result goes to the first 16 of their own columns.
#include "xattn.cuh"

namespace nvfp4 {
namespace xattn {

constexpr int kBwdThreads = 640;
constexpr int kBwdWarps = 16;                 // on a tile
constexpr int kBwdCols = 32;                  // columns of one
// Of eight pairs of dK/dV's exponentials, on the FMA pipes: a step of 128 x 128, d = 128, takes 3150 to 3300 cycles with 4,
// 3410 with none (they come between two hand-overs).  dQ's run beside its products: 2590 with 4, 2510 to 2580 with none.
constexpr int kPolyPairs = 4;
constexpr int kBwdRegsLow = 64;               // 128 x 64 + 512 x 104 <= 640 x 96
constexpr int kBwdRegsHigh = 104;
static_assert(128 * kBwdRegsLow + 512 * kBwdRegsHigh <= kBwdThreads * 96, "register split exceeds the launch budget");

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

// The packed values of 32 columns start where those columns did: an A operand of two steps a group.
constexpr int kPackedGroup = kBwdCols / 16;

// ------------------------------------------------------------------ D
constexpr int kDeltaThreads = 256;
constexpr int kDeltaRows = 4;                 // rows of 16 lanes, each at once

__global__ void __launch_bounds__(kDeltaThreads) delta_kernel(const nvfp4_heads grad_out, const nvfp4_heads out, float* delta,
                                                              int rows, int Lq, int H, int d) {
    const int lane = threadIdx.x & 15;
    const uint32_t first = blockIdx.x * (kDeltaThreads / 16 * kDeltaRows) + threadIdx.x / 16;
    uint4 a[kDeltaRows], b[kDeltaRows];
    int64_t at[kDeltaRows];
#pragma unroll
    for (int i = 0; i < kDeltaRows; ++i) {
        const uint32_t r = first + i * (kDeltaThreads / 16);         // (b, l, h), heads innermost
        a[i] = b[i] = make_uint4(0, 0, 0, 0);
        at[i] = -1;
        if (r >= (uint32_t)rows) continue;
        const uint32_t bl = r / (uint32_t)H, h = r - bl * H, bb = bl / (uint32_t)Lq, l = bl - bb * Lq;
        at[i] = ((int64_t)bb * H + h) * Lq + l;
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
    MapAxes aq, ag, ak, av, ad;
    nvfp4_heads dq;
    const float* lse;
    float* delta;                             // D (out for samples of one key tile)
    const int32_t* kv_lens;
    float c, scale;                           // scale * log2(e), scale
    int H, Hkv, Lq, Lk, d;
    int group, qtiles, items;
    int chunks, qbufs, kbufs, vbufs;
    bool zeros;                               // dQ of samples without keys is this launch's
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

// The next item at or after `it` (in this block's stride) that the kernel takes: ONE those of one step, the other of more.
template <bool ONE>
__device__ __forceinline__ int dq_next(const DqParams& p, int it, DqItem& item) {
    for (; it < p.items; it += gridDim.x) {
        item = dq_item(p, it);
        if (ONE ? item.steps == 1 : item.steps > 1) break;
    }
    return it;
}

// A walk over the steps of this block's items, in order.
template <bool ONE>
struct DqWalk {
    int it, j;
    DqItem item;
    __device__ void start(const DqParams& p) {
        j = 0;
        it = dq_next<ONE>(p, blockIdx.x, item);
    }
    __device__ bool valid(const DqParams& p) const { return it < p.items; }
    __device__ void next(const DqParams& p) {
        if (++j == item.steps) {
            j = 0;
            it = dq_next<ONE>(p, it + gridDim.x, item);
        }
    }
};

// D of a row whose keys are all in this tile, sum P dP, which unlike sum dO O has no rounding of O in it (with few keys
// dP is close to D, and that rounding the larger part of dS's error): each of the four warps of a row adds its n
// columns, p the P of them, the sums meet in d_part.  Out of line, so that its registers are not the main loop's.
// (d_part is written again after the next dP, which comes after every warp has used this one's D.)
__device__ __noinline__ bool row_d(const float* p, uint32_t dp_at, int n, int g, int r, uint64_t* bar, uint32_t parity,
                                   float (*d_part)[kRows], const WaitCtx& wc, float* d) {
    float sum[2] = {0.0f, 0.0f};
    if (n > 0) {
        uint32_t dp[32];
        tmem_ld_32x32b_x32(dp_at, dp);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n) sum[i & 1] = fmaf(p[i], __uint_as_float(dp[i]), sum[i & 1]);
    }
    d_part[g][r] = sum[0] + sum[1];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
    if (!warp_wait(bar, parity, wc)) return false;
    *d = ((d_part[0][r] + d_part[1][r]) + d_part[2][r]) + d_part[3][r];
    return true;
}

constexpr int kMaxQ = 4, kMaxK = 4, kMaxV = 4;
constexpr uint32_t kDqS = 0, kDqP = 256, kDqO = 384;      // S: [128 (s & 1), + 128); dP; dQ

// ONE: the samples of one key tile, whose D is formed here; the others' comes from delta_kernel.
template <bool ONE>
__global__ void __launch_bounds__(kBwdThreads, 1)
xattn_dq_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_g,
                const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                const __grid_constant__ CUtensorMap tmap_dq, const DqParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t q_full[kMaxQ], q_empty[kMaxQ], k_full[kMaxK], k_empty[kMaxK], v_full[kMaxV], v_empty[kMaxV];
    __shared__ __align__(8) uint64_t s_full[2], dp_full, ds_ready, dq_full, drain;
    __shared__ __align__(8) uint64_t d_bar[4];
    __shared__ float d_part[4][kRows];                      // [column group][row]
    __shared__ uint32_t k_info[kMaxK], tmem_base_sh;
    __shared__ int abort_sh;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int tile_bytes = p.chunks * kChunk;
    uint8_t* k_tiles = smem + p.qbufs * tile_bytes;
    uint8_t* v_tiles = k_tiles + p.kbufs * tile_bytes;
    WaitCtx wc{&abort_sh, p.dev_status};
    if ((smem_u32(smem) & 1023u) != 0u) {           // the swizzled layouts need it; the declaration asks for it
        if (p.dev_status) *p.dev_status = (int)NVFP4_ERR_MISALIGNED;
        return;
    }

    if (ONE && !p.zeros) {                          // beside a launch for longer samples: often there is nothing to do
        int any = 0;
        const int samples = p.items / (p.H * p.qtiles);
        for (int b = threadIdx.x; b < samples; b += kBwdThreads) {
            const int keys = keys_of(p.kv_lens, b, p.Lk);
            any |= keys > 0 && keys <= kRows;
        }
        if (!__syncthreads_or(any)) return;
    }

    if (threadIdx.x == 0) {
        abort_sh = 0;
        for (int i = 0; i < kMaxQ; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1 + kBwdWarps);      // the tile's last product, the warps
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
        mbar_init(&ds_ready, kBwdWarps);
        mbar_init(&dq_full, 1);
        for (int i = 0; i < 4; ++i) mbar_init(&d_bar[i], 4);
        mbar_init(&drain, 1);
        fence_barrier_init();
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_g);
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
        tma_prefetch_desc(&tmap_dq);
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
            DqWalk<ONE> w;
            bool ok = true;
            auto load = [&](TileRing& ring, uint64_t* full, uint64_t* empty, uint8_t* tiles, const CUtensorMap* map, int h, int l,
                            int b, uint32_t* info, uint32_t value) {
                if (!warp_wait(&empty[ring.slot], ring.phase ^ 1u, wc)) return false;
                if (lane == 0) {
                    if (info) info[ring.slot] = value;
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
                ok = (w.j > 0 || load(rq, q_full, q_empty, smem, &tmap_q, i.h * p.aq.h, i.q0, i.b * p.aq.b, nullptr, 0)) &&
                     load(rk, k_full, k_empty, k_tiles, &tmap_k, hk * p.ak.h, w.j * kRows, i.b * p.ak.b, k_info,
                          step_info(i.keys, p.Lk, w.j, i.steps, false)) &&
                     (w.j > 0 || load(rq, q_full, q_empty, smem, &tmap_g, i.h * p.ag.h, i.q0, i.b * p.ag.b, nullptr, 0)) &&
                     load(rv, v_full, v_empty, v_tiles, &tmap_v, hk * p.av.h, w.j * kRows, i.b * p.av.b, nullptr, 0);
            }
            if (ok && warp_wait(&k_empty[rk.slot], rk.phase ^ 1u, wc) && lane == 0) {
                k_info[rk.slot] = 0;
                mbar_arrive(&k_full[rk.slot]);
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
            uint32_t s_at = 0, done = 0;                         // S products, dS so far
            int q_slot = 0, g_slot = 0;
            bool ok = true;

            // S of the step whose K tile comes next; returns its description
            auto issue_s = [&]() -> uint32_t {
                if (!(ok = warp_wait(&k_full[ks.slot], ks.phase, wc))) return 0;
                const uint32_t info = k_info[ks.slot];
                if (info == 0) return 0;
                if (info & kInfoFirst) {
                    q_slot = qs.slot;
                    if (!(ok = warp_wait(&q_full[qs.slot], qs.phase, wc))) return 0;
                    qs.next();
                    qs.next();
                }
                tc_fence_after();
                product_kk(tmem + kDqS + (s_at & 1u) * 128, q_sm + q_slot * tile_bytes, k_sm + ks.slot * tile_bytes,
                           idesc_kk((int)((info & kInfoKeys) + 15) & ~15), dsteps);
                commit(&s_full[s_at & 1u]);
                if (info & kInfoLast) commit(&q_empty[q_slot]);
                ks.next();
                ++s_at;
                return info;
            };
            auto issue_dp = [&](uint32_t info) {
                if (info & kInfoFirst) {
                    g_slot = qp.slot;
                    if (!warp_wait(&q_full[qp.slot], qp.phase, wc)) return false;
                    qp.next();
                    qp.next();
                }
                if (!warp_wait(&v_full[rv.slot], rv.phase, wc)) return false;
                tc_fence_after();
                product_kk(tmem + kDqP, q_sm + g_slot * tile_bytes, v_sm + rv.slot * tile_bytes,
                           idesc_kk((int)((info & kInfoKeys) + 15) & ~15), dsteps);
                commit(&dp_full);
                commit(&v_empty[rv.slot]);
                if (info & kInfoLast) commit(&q_empty[g_slot]);
                rv.next();
                return true;
            };

            uint32_t cur = issue_s(), nxt = 0;
            if (cur) ok = issue_dp(cur);
            if (ok && cur) nxt = issue_s();
            while (ok && cur) {
                const int n = (int)(cur & kInfoKeys);
                if (!(ok = warp_wait(&ds_ready, done & 1u, wc))) break;
                if (nxt && !(ok = issue_dp(nxt))) break;
                if (cur & kInfoZero) zero_rest(k_tiles + kq.slot * tile_bytes, n, p.chunks, lane);   // S of the step is done
                tc_fence_after();
                product_tmem<kPackedGroup>(tmem + kDqO, tmem + kDqS + (done & 1u) * 128, k_sm + kq.slot * tile_bytes,
                                           idesc_o, (n + 15) >> 4, (cur & kInfoFirst) == 0);
                commit(&k_empty[kq.slot]);
                if (cur & kInfoLast) commit(&dq_full);
                kq.next();
                ++done;
                cur = nxt;
                if (nxt) nxt = issue_s();
            }
            commit(&drain);
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
        const uint32_t tbase = tmem + lane_base + g * kBwdCols;
        uint32_t step = 0, outs = 0, singles = 0;
        bool ok = true;

        auto row_at = [&](const DqItem& i) {
            return static_cast<uint16_t*>(p.dq.data) + (int64_t)i.b * p.dq.batch_stride + (int64_t)(i.q0 + r) * p.dq.token_stride +
                   (int64_t)i.h * p.dq.head_stride + g * kBwdCols;
        };
        const int cols = min(max(p.d - g * kBwdCols, 0), kBwdCols);        // of d this warp reads out
        // Q and dO tiles of the items in the order of their loads: the warps let go of a Q tile at once,
        // of a dO tile when dQ has gone out from it
        int q_slot = 0, g_slot = 1 % p.qbufs, from = -1;
        uint8_t* const staged = smem + (g * 4 + quarter) * 2048;           // + slot: 32 rows of 64 bytes, 64-byte swizzle
        auto read_out = [&](const DqItem& i) {
            if (!warp_wait(&dq_full, outs & 1u, wc)) return false;
            ++outs;
            if (cols > 0) {
                tc_fence_after();
                uint32_t o[32];
                tmem_ld_32x32b_x32(tbase + kDqO, o);
                tmem_ld_wait();
                uint8_t* dst = staged + from * tile_bytes;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t w[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        w[u] = pack_bf16(__uint_as_float(o[8 * e + 2 * u]) * p.scale, __uint_as_float(o[8 * e + 2 * u + 1]) * p.scale);
                    *reinterpret_cast<uint4*>(dst + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (i.q0 + quarter * 32 < p.Lq)
                        tma_store_4d(&tmap_dq, dst, g * kBwdCols, i.h * p.ad.h, i.q0 + quarter * 32, i.b * p.ad.b);
                    bulk_commit_group();
                }
            }
            return true;
        };
        auto release = [&]() {                      // the dO tile, once dQ has been read from it
            if (lane == 0) {
                bulk_wait_group_read<0>();
                mbar_arrive(&q_empty[from]);
            }
            from = -1;
            __syncwarp();
        };

        // the next item's lse (times log2(e)) and D are on their way while this one's steps run
        auto fetch = [&](int it, DqItem& i, float& l, float& delta) {
            i = dq_item(p, it);
            const int64_t at = ((int64_t)i.b * p.H + i.h) * p.Lq + i.q0 + r;
            const bool have = i.q0 + r < p.Lq;
            l = have ? __ldg(p.lse + at) : INFINITY;
            delta = have && !ONE ? __ldg(p.delta + at) : 0.0f;
        };
        DqItem prev, item, following;
        float lse = 0.0f, dl = 0.0f, next_lse = 0.0f, next_dl = 0.0f;
        bool pending = false;
        if ((int)blockIdx.x < p.items) fetch(blockIdx.x, item, lse, dl);
        for (int it = blockIdx.x; ok && it < p.items; it += gridDim.x, item = following, lse = next_lse, dl = next_dl) {
            if (it + (int)gridDim.x < p.items) fetch(it + gridDim.x, following, next_lse, next_dl);
            if (item.steps == 0) {
                if (p.zeros && item.q0 + r < p.Lq)
                    for (int i = 0; i < cols; i += 8) *reinterpret_cast<uint4*>(row_at(item) + i) = make_uint4(0, 0, 0, 0);
                continue;
            }
            if (ONE != (item.steps == 1)) continue;
            const float lse2 = lse * kLog2e;
            for (int j = 0; j < item.steps; ++j, ++step) {
                const int n = min(max(item.keys - j * kRows - g * kBwdCols, 0), kBwdCols);      // this warp's keys
                const uint32_t ts = tbase + kDqS + (step & 1u) * 128, tp = tbase + kDqP;
                if (!(ok = warp_wait(&s_full[step & 1u], (step >> 1) & 1u, wc))) break;
                tc_fence_after();
                if (j == 0 && lane == 0) mbar_arrive(&q_empty[q_slot]);
                uint32_t v[32];
                if (n > 0) {
                    tmem_ld_32x32b_x32(ts, v);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const F2 x = fma2({__uint_as_float(v[i]), __uint_as_float(v[i + 1])}, {p.c, p.c}, {-lse2, -lse2});
                    v[i] = __float_as_uint(ex2(x.x));
                    v[i + 1] = __float_as_uint(ex2(x.y));
                }
                if (pending) {
                    if (!(ok = read_out(prev))) break;
                    pending = false;
                }
                if (!(ok = warp_wait(&dp_full, step & 1u, wc))) break;
                tc_fence_after();
                if (ONE) {
                    float copy[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) copy[i] = __uint_as_float(v[i]);
                    if (!(ok = row_d(copy, tp, n, g, r, &d_bar[quarter], singles & 1u, d_part, wc, &dl))) break;
                    ++singles;
                    if (g == 0 && item.q0 + r < p.Lq) p.delta[((int64_t)item.b * p.H + item.h) * p.Lq + item.q0 + r] = dl;
                }
                if (n > 0) {
                    uint32_t dp[32], w[16];
                    tmem_ld_32x32b_x32(tp, dp);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const F2 x = mul2(add2({__uint_as_float(dp[i]), __uint_as_float(dp[i + 1])}, {-dl, -dl}),
                                          {__uint_as_float(v[i]), __uint_as_float(v[i + 1])});
                        // keys past the length: zero, whatever was computed there
                        w[i / 2] = pack_bf16(i < n ? x.x : 0.0f, i + 1 < n ? x.y : 0.0f);
                    }
                    tmem_st_x16(ts, w);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ds_ready);
                if (from >= 0 && !pending) release();
            }
            prev = item;
            pending = ok;
            from = g_slot;
            q_slot = (q_slot + 2) % p.qbufs;
            g_slot = (g_slot + 2) % p.qbufs;
        }
        if (ok && pending && read_out(prev)) release();
        if (lane == 0) bulk_wait_group_read<0>();
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
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
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
        mbar_init(&p_ready, kBwdWarps);
        mbar_init(&ds_ready, kBwdWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&st_full[i], 32);
            mbar_init(&st_empty[i], kBwdWarps);
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
            // S^T or dP^T of a step with n queries: rows = keys, columns = queries
            auto scores = [&](int n, TileRing& ring, uint32_t a_sm, uint32_t col, uint64_t* bar) {
                if (!warp_wait(&qg_full[ring.slot], ring.phase, wc)) return false;
                tc_fence_after();
                product_kk(tmem + col, a_sm, qg_sm + ring.slot * tile_bytes, idesc_kk((n + 15) & ~15), dsteps);
                commit(bar);
                ring.next();
                ring.next();
                return true;
            };
            // dV or dK += (P^T or dS^T) (dO or Q)
            auto update = [&](int n, TileRing& ring, uint32_t a, uint32_t col, bool accumulate) {
                tc_fence_after();
                product_tmem<kPackedGroup>(tmem + col, tmem + a, qg_sm + ring.slot * tile_bytes, idesc_o, (n + 15) >> 4,
                                           accumulate);
                commit(&qg_empty[ring.slot]);
                ring.next();
                ring.next();
            };
            int q0 = (first % p.qtiles) * kRows;                 // first query of the step
            int n = min(p.Lq - q0, kRows);
            bool ok = warp_wait(&k_full, 0, wc) && scores(n, rs, k_sm, kKvS, &s_full) && warp_wait(&v_full, 0, wc) &&
                      scores(n, rp, v_sm, kKvP, &dp_full);
            uint32_t ph = 0;
            for (int t = first; ok && t < last; ++t, ph ^= 1u) {
                q0 = q0 + kRows < p.Lq ? q0 + kRows : 0;
                const int n2 = min(p.Lq - q0, kRows);            // of the next step
                if (!(ok = warp_wait(&p_ready, ph, wc))) break;
                update(n, rv, kKvS, kKvV, t > first);
                if (t + 1 < last && !(ok = scores(n2, rs, k_sm, kKvS, &s_full))) break;
                if (!(ok = warp_wait(&ds_ready, ph, wc))) break;
                update(n, rk, kKvP, kKvK, t > first);
                if (t + 1 < last) ok = scores(n2, rp, v_sm, kKvP, &dp_full);
                n = n2;
            }
            commit(&drain);
            __syncwarp();
            int dummy = 0;
            WaitCtx w2{&dummy, p.dev_status};
            mbar_wait(&drain, 0, w2);
        } else if (warp == 2) {
            // -------------------------------------------------------- -lse (times log2(e)) and -D of the steps' queries
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
                    l[i] = have ? -(__ldg(p.lse + at + lane + 32 * i) * kLog2e) : -INFINITY;
                    dl[i] = have ? -__ldg(p.delta + at + lane + 32 * i) : 0.0f;
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
        const uint32_t ts = tmem + lane_base + kKvS + g * kBwdCols, tp = tmem + lane_base + kKvP + g * kBwdCols;
        bool ok = true;
        for (int t = first; t < last; ++t) {
            const int s = (t - first) & 1;
            const uint32_t ph = (uint32_t)(t - first) & 1u;
            const float4* lse4 = reinterpret_cast<const float4*>(&st_lse[s][g * kBwdCols]);
            const float4* del4 = reinterpret_cast<const float4*>(&st_delta[s][g * kBwdCols]);
            if (!(ok = warp_wait(&st_full[s], ((uint32_t)(t - first) >> 1) & 1u, wc) && warp_wait(&s_full, ph, wc))) break;
            tc_fence_after();
            uint32_t v[32], w[16];
            tmem_ld_32x32b_x32(ts, v);
            tmem_ld_wait();
            // columns past the last query hold anything: -lse = -infinity alone would leave NaN there
            const int nq = p.Lq - (t % p.qtiles) * kRows - g * kBwdCols;
            if (nq < kBwdCols) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (i >= nq) v[i] = 0;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 l = lse4[i];                            // kept negated
                const F2 x = ex2_pair<kPolyPairs>(
                    fma2({__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1])}, {p.c, p.c}, {l.x, l.y}), 2 * i);
                const F2 y = ex2_pair<kPolyPairs>(
                    fma2({__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])}, {p.c, p.c}, {l.z, l.w}), 2 * i + 1);
                v[4 * i] = __float_as_uint(x.x);
                v[4 * i + 1] = __float_as_uint(x.y);
                v[4 * i + 2] = __float_as_uint(y.x);
                v[4 * i + 3] = __float_as_uint(y.y);
                w[2 * i] = pack_bf16(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]));
                w[2 * i + 1] = pack_bf16(__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
            }
            tmem_st_x16(ts, w);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready);

            if (!(ok = warp_wait(&dp_full, ph, wc))) break;
            tc_fence_after();
            uint32_t dp[32];
            tmem_ld_32x32b_x32(tp, dp);
            tmem_ld_wait();
            if (nq < kBwdCols) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (i >= nq) dp[i] = 0;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 dl = del4[i];                           // kept negated
                const F2 x = mul2(add2({__uint_as_float(dp[4 * i]), __uint_as_float(dp[4 * i + 1])}, {dl.x, dl.y}),
                                  {__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1])});
                const F2 y = mul2(add2({__uint_as_float(dp[4 * i + 2]), __uint_as_float(dp[4 * i + 3])}, {dl.z, dl.w}),
                                  {__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])});
                w[2 * i] = pack_bf16(x.x, x.y);
                w[2 * i + 1] = pack_bf16(y.x, y.y);
            }
            tmem_st_x16(tp, w);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&st_empty[s]);
                mbar_arrive(&ds_ready);
            }
        }
        // the sums: this thread's key, 32 of the d columns
        const int cols = min(max(p.d - g * kBwdCols, 0), kBwdCols);
        if (ok && warp_wait(&drain, 0, wc) && cols > 0) {
            tc_fence_after();
#pragma unroll 1
            for (int o = 0; o < 2; ++o) {
                const float f = o == 0 ? p.scale : 1.0f;
                const nvfp4_heads& t = o == 0 ? p.dk : p.dv;
                uint32_t x[32];
                tmem_ld_32x32b_x32(tmem + lane_base + (o == 0 ? kKvK : kKvV) + g * kBwdCols, x);
                tmem_ld_wait();
                if (p.partial) {
                    float* part = p.partial + (((int64_t)split * (gridDim.x / p.splits) + unit) * 2 + o) * p.d * kRows +
                                  ((int64_t)g * (kBwdCols / 4) * kRows + r) * 4;
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        if (e >= cols) break;
                        *reinterpret_cast<uint4*>(part + e * kRows) = make_uint4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                    }
                } else if (k0 + r < p.Lk) {
                    const bool valid = k0 + r < keys;
                    uint16_t* dst = static_cast<uint16_t*>(t.data) + (int64_t)b * t.batch_stride +
                                    (int64_t)(k0 + r) * t.token_stride + (int64_t)hk * t.head_stride + g * kBwdCols;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        if (e >= cols) break;
                        uint32_t y[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            y[u] = valid ? pack_bf16(__uint_as_float(x[e + 2 * u]) * f, __uint_as_float(x[e + 2 * u + 1]) * f) : 0u;
                        *reinterpret_cast<uint4*>(dst + e) = make_uint4(y[0], y[1], y[2], y[3]);
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
// The SMs of the GPUs that the library runs on.  The plan sizes the workspace, which is asked for by sizes alone, on hosts
// without a GPU too, and has to be the same wherever the call then runs: it does not ask the device.
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

// Dynamic shared memory a launch may ask for.  Always the same limit: it belongs to the kernel, and another thread may be
// about to launch with more.
cudaError_t prepare_kernel(const void* kernel, int most) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
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
    CUtensorMap mq{}, mg{}, mk{}, mv{}, md{};
    MapAxes aq{}, ag{}, ak{}, av{}, ad{};
    if (a.Lq > 0 && a.Lk > 0 &&
        (!make_heads_map(&mq, a.q, a.B, a.Lq, a.H, a.d, kRows, &aq) || !make_heads_map(&mg, a.grad_out, a.B, a.Lq, a.H, a.d, kRows, &ag) ||
         !make_heads_map(&mk, a.k, a.B, a.Lk, a.Hkv, a.d, kRows, &ak) || !make_heads_map(&mv, a.v, a.B, a.Lk, a.Hkv, a.d, kRows, &av) ||
         !make_heads_map(&md, a.dq, a.B, a.Lq, a.H, a.d, 32, &ad, kBwdCols)))
        return cudaErrorInvalidValue;
    cudaError_t e;
    int launches = 0;
    if (a.Lq > 0) {
        if (ktiles > 1) {
            const int64_t rows = (int64_t)a.B * a.Lq * a.H;
            const int64_t per = kDeltaThreads / 16 * kDeltaRows;
            delta_kernel<<<(unsigned)((rows + per - 1) / per), kDeltaThreads, 0, stream>>>(a.grad_out, a.out, delta, (int)rows,
                                                                                           a.Lq, a.H, a.d);
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
            ++launches;
        }
        DqParams p{aq, ag, ak, av, ad, a.dq, a.lse, delta, a.kv_lens, a.scale * kLog2e, a.scale, a.H, a.Hkv, a.Lq, a.Lk, a.d,
                   a.H / a.Hkv, qtiles, a.B * a.H * qtiles, chunks, chunks == 1 ? 4 : 3, chunks == 1 ? 4 : 3, chunks == 1 ? 4 : 1,
                   true, a.dev_status};
        const int smem = (p.qbufs + p.kbufs + p.vbufs) * tile_bytes;
        // samples of several key tiles, then (where lengths tell) those of one
        for (int pass = 0; pass < 2; ++pass) {
            const bool one = pass == 1;
            if (one ? ktiles > 1 && !a.kv_lens : ktiles <= 1) continue;
            p.zeros = one == (ktiles <= 1);
            const auto kernel = one ? xattn_dq_kernel<true> : xattn_dq_kernel<false>;
            if ((e = prepare_kernel(reinterpret_cast<const void*>(kernel), 14 * kChunk)) != cudaSuccess) return e;
            kernel<<<p.items < num_sms ? p.items : num_sms, kBwdThreads, smem, stream>>>(mq, mg, mk, mv, md, p);
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
            ++launches;
        }
    }
    if (plan.units > 0 && plan.splits > 0) {
        DkvParams p{aq, ag, ak, av, a.dk, a.dv, a.lse, delta, a.kv_lens, partial, a.scale * kLog2e, a.scale, a.H, a.Hkv, a.Lq, a.Lk,
                    a.d, a.H / a.Hkv, qtiles, ktiles, (int)plan.steps, plan.splits, chunks, chunks == 1 ? 8 : 4, a.dev_status};
        const int smem = (2 + p.qbufs) * tile_bytes + 1024;
        if ((e = prepare_kernel(reinterpret_cast<const void*>(xattn_dkv_kernel), 12 * kChunk + 1024)) != cudaSuccess) return e;
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
