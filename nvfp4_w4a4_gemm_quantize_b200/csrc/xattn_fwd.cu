// xattn_fwd.cu -- attention to an encoder's states of another length, forward
// (nvfp4_cross_attention), for more than a few queries.
//
//   S = Q K^T, P = 2^(c S - m) with c = scale log2(e), O = P V / sum P
// with an online softmax: m is a running reference maximum, sum P and O are
// rescaled when it moves.  m moves only when a tile exceeds it by more than 8
// (P stays below 2^8; nothing is lost in FP32), so most tiles touch O only
// through the tensor cores.
//
// Persistent, one CTA per SM.  A work item is a pair of 128-query tiles A and B
// that read the same keys: consecutive tiles of the query heads of one sample's
// key / value head (so heads that share one pair up too; a last odd tile runs
// alone).  Keys come in tiles of 128; the last one computes only as many as it
// holds, rounded up to 16.
// TMEM (512 columns): S_A, S_B, O_A, O_B.  P overwrites its S as packed bf16
// and is the A operand of the second product from there.  One warp issues every
// product, in the order S_A S_B | P V_A, next S_A | P V_B, next S_B | ...: the
// tensor core works for one tile while the other's softmax runs, and S of the
// next tile needs no barrier of its own, since the tensor core takes it after
// the product that read P.  The order runs on across work items.
// Warps: 0 loads (four rotating Q tiles, a ring of K and V tiles), 1 issues
// and owns TMEM, 4-7 and 8-11 softmax and output of A and B, a thread per row.
// The output goes out by TMA from the item's own Q tile: written from the
// registers, a row per thread, it took 6400 cycles an item (a 128-byte line per
// lane and store), as long as two steps.  It is read out once the next item's
// first P is stored, so that the wait for the last product has gone by.
// P is rounded to bf16 for P V, as the tensor core wants both operands in one type
// and V is bf16: the output is 2.2e-3 off the formula in 64 bits (relative, in the
// norm) where FP32 arithmetic rounded once is 1.7e-3; P as TF32 would halve the rate.
// Bound by a tile's chain, softmax -> P V -> next S -> softmax: a tile has one S,
// and P takes its place.  A step (128 keys of a pair of tiles) takes 3550 to 3600
// cycles, for heads of 72 as for 128 (the slope over 512 to 2048 keys): its
// exponentials take 2048 of the hardware's unit and its products at d = 128 as much
// of the tensor core, but those of the two tiles overlap in part, each hand-over
// between warps and tensor core takes 200 to 300, and the issuing warp, next to busy
// ones, needs about as long for a product as the tensor core.  An item's start and
// end come to 5000 to 7000 on top: 4900 a step for items of four.
// B200, 32768 queries x 512 states, 24 heads of 128: 214 us (963 TFLOP/s) in a burst
// at 1965 MHz, 220 to 240 sustained, where the 1000 W limit holds 1.73 GHz.
#include "xattn.cuh"

namespace nvfp4 {
namespace xattn {

constexpr int kThreads = 384;
constexpr int kQBufs = 4;                     // two items' tiles: an output leaves from its own during the next item's steps
static_assert(kQBufs >= 4, "an item would wait for the tiles of the one before it, and that one for this item");
constexpr int kMaxRing = 12;
constexpr int kRegsLow = 88;                  // 128 x 88 + 256 x 208 <= 384 x 168
constexpr int kRegsHigh = 208;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= kThreads * 168, "register split exceeds the launch budget");

constexpr uint32_t kColS = 0;                 // S_g (and P_g): [128 g, 128 g + 128)
constexpr uint32_t kColO = 256;               // O_g: [256 + 128 g, 384 + 128 g)

struct FwdParams {
    MapAxes aq, ak, av, ao;
    nvfp4_heads out;
    float* lse;
    const int32_t* kv_lens;
    float c;                                  // scale * log2(e)
    int H, Hkv, Lq, Lk, d;
    int group, qtiles, tiles, pairs, items;   // query heads per kv head, tiles of a head, of a kv head, pairs of those
    int chunks, ring;
    int* dev_status;
};

// Work item: sample, kv head, first tile; its key count.
struct Item {
    int b, hk, tile, keys, steps;
    bool two;
};

__device__ __forceinline__ Item item_of(const FwdParams& p, int it) {
    Item r;
    const int bh = it / p.pairs;
    r.tile = (it - bh * p.pairs) * 2;
    r.b = bh / p.Hkv;
    r.hk = bh - r.b * p.Hkv;
    r.two = r.tile + 1 < p.tiles;
    r.keys = keys_of(p.kv_lens, r.b, p.Lk);
    r.steps = (r.keys + kRows - 1) / kRows;
    return r;
}

// Head and first query of tile g of an item.
__device__ __forceinline__ void tile_place(const FwdParams& p, const Item& i, int g, int& head, int& q0) {
    const int t = i.tile + g, in_group = t / p.qtiles;
    head = i.hk * p.group + in_group;
    q0 = (t - in_group * p.qtiles) * kRows;
}

// The next item at or after `it` (in this CTA's stride) that has keys.
__device__ __forceinline__ int next_item(const FwdParams& p, int it, Item& item) {
    for (; it < p.items; it += gridDim.x) {
        item = item_of(p, it);
        if (item.steps > 0) break;
    }
    return it;
}

// A ring position and its phase parity.
struct RingAt {
    int slot;
    uint32_t phase;
    __device__ void advance(int by, int n) {
        slot += by;
        if (slot >= n) {
            slot -= n;
            phase ^= 1u;
        }
    }
};

__global__ void __launch_bounds__(kThreads, 1)
xattn_fwd_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                 const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_o, const FwdParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t q_full[kQBufs], q_empty[kQBufs], kv_full[kMaxRing], kv_empty[kMaxRing];
    __shared__ __align__(8) uint64_t s_full[2], p_full[2], o_full[2], drain;
    __shared__ uint32_t kv_info[kMaxRing], tmem_base_sh;
    __shared__ int abort_sh;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tile_bytes = p.chunks * kChunk;
    uint8_t* ring = smem + kQBufs * tile_bytes;
    WaitCtx wc{&abort_sh, p.dev_status};

    if (threadIdx.x == 0) {
        abort_sh = 0;
        for (int i = 0; i < kQBufs; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 5);              // the tile's last S product, the group's warps
        }
        for (int i = 0; i < kMaxRing; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);             // the last product that reads it
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&s_full[g], 1);
            mbar_init(&p_full[g], 4);               // the group's warps
            mbar_init(&o_full[g], 1);
        }
        mbar_init(&drain, 1);
        fence_barrier_init();
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
        tma_prefetch_desc(&tmap_o);
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
        regs_dec<kRegsLow>();
        if (warp == 0) {
            // -------------------------------------------------------- loads, in the order the issuer consumes them
            RingAt at{0, 0}, qa{0, 0};
            Item item;
            bool ok = true;
            auto load_q = [&](int g) {
                if (!warp_wait(&q_empty[qa.slot], qa.phase ^ 1u, wc)) return false;
                if (elect_one()) {
                    int head, q0;
                    tile_place(p, item, g, head, q0);
                    mbar_arrive_expect_tx(&q_full[qa.slot], (uint32_t)tile_bytes);
                    load_tile(smem + qa.slot * tile_bytes, &tmap_q, &q_full[qa.slot], p.chunks, kChunk, head * p.aq.h, q0,
                              item.b * p.aq.b);
                }
                __syncwarp();
                qa.advance(1, kQBufs);
                return true;
            };
            auto load_kv = [&](const CUtensorMap* map, const MapAxes& axes, int j) {
                if (!warp_wait(&kv_empty[at.slot], at.phase ^ 1u, wc)) return false;
                if (lane == 0) {
                    kv_info[at.slot] = step_info(item.keys, p.Lk, j, item.steps, item.two);
                    mbar_arrive_expect_tx(&kv_full[at.slot], (uint32_t)tile_bytes);
                    load_tile(ring + at.slot * tile_bytes, map, &kv_full[at.slot], p.chunks, kChunk, item.hk * axes.h,
                              j * kRows, item.b * axes.b);
                }
                __syncwarp();
                at.advance(1, p.ring);
                return true;
            };
            for (int it = next_item(p, blockIdx.x, item); ok && it < p.items; it = next_item(p, it + gridDim.x, item)) {
                ok = load_q(0) && load_kv(&tmap_k, p.ak, 0) && (!item.two || load_q(1)) && load_kv(&tmap_v, p.av, 0);
                for (int j = 1; ok && j < item.steps; ++j) ok = load_kv(&tmap_k, p.ak, j) && load_kv(&tmap_v, p.av, j);
            }
            if (ok && warp_wait(&kv_empty[at.slot], at.phase ^ 1u, wc) && lane == 0) {
                kv_info[at.slot] = 0;                            // no more steps
                mbar_arrive(&kv_full[at.slot]);
            }
            __syncwarp();
            // a block that gave up still waits for its loads in flight
            if (!ok && lane == 0) {
                int dummy = 0;
                WaitCtx w2{&dummy, p.dev_status};
                RingAt a = at;
                for (int i = 0; i < p.ring; ++i) {
                    a.slot = a.slot == 0 ? p.ring - 1 : a.slot - 1;
                    if (a.slot == p.ring - 1) a.phase ^= 1u;
                    if (i < p.ring) mbar_wait_limit(&kv_full[a.slot], a.phase, w2, 1000000);
                }
                for (int i = 0; i < kQBufs; ++i) mbar_wait_limit(&q_full[i], i < qa.slot ? qa.phase : qa.phase ^ 1u, w2, 1000000);
            }
        } else if (warp == 1) {
            // -------------------------------------------------------- products
            const uint32_t q_sm = smem_u32(smem), ring_sm = smem_u32(ring);
            const int dsteps = (p.d + 15) >> 4;
            const uint32_t idesc_o = idesc_kmn(dsteps * 16);
            RingAt kat{0, 0}, vat{1, 0};            // K and V tiles alternate in the ring
            RingAt qat{0, 0};
            uint32_t uses[2] = {0, 0};              // tiles of each group so far
            int q_buf[2] = {0, 0};
            bool ok = true;

            // the description of the step whose K tile comes next
            auto describe = [&]() -> uint32_t {
                if (!(ok = warp_wait(&kv_full[kat.slot], kat.phase, wc))) return 0;
                return kv_info[kat.slot];
            };
            // S_g of that step; the last product on the K tile frees it
            auto issue_s = [&](uint32_t info, int g) {
                if (info & kInfoFirst) {
                    q_buf[g] = qat.slot;
                    if (!warp_wait(&q_full[qat.slot], qat.phase, wc)) return false;
                    qat.advance(1, kQBufs);
                }
                tc_fence_after();
                product_kk(tmem + kColS + g * 128, q_sm + q_buf[g] * tile_bytes, ring_sm + kat.slot * tile_bytes,
                           idesc_kk((int)((info & kInfoKeys) + 15) & ~15), dsteps);
                commit(&s_full[g]);
                if (info & kInfoLast) commit(&q_empty[q_buf[g]]);
                if (g == 1 || !(info & kInfoTwo)) {
                    commit(&kv_empty[kat.slot]);
                    kat.advance(2, p.ring);
                }
                return true;
            };

            uint32_t cur = describe();
            if (cur) ok = issue_s(cur, 0) && (!(cur & kInfoTwo) || issue_s(cur, 1));
            while (ok && cur) {
                const int n = (int)(cur & kInfoKeys);
                const uint32_t vt = ring_sm + vat.slot * tile_bytes;
                uint32_t nxt = 0;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    if (g == 1 && !(cur & kInfoTwo)) continue;
                    // (an item's first P comes after the previous item's O_g has been read out)
                    ok = ok && warp_wait(&p_full[g], uses[g] & 1u, wc) && (g == 1 || warp_wait(&kv_full[vat.slot], vat.phase, wc));
                    if (!ok) break;
                    ++uses[g];
                    if (g == 0 && (cur & kInfoZero)) zero_rest(ring + vat.slot * tile_bytes, n, p.chunks, lane);
                    tc_fence_after();
                    product_tmem<8>(tmem + kColO + g * 128, tmem + kColS + g * 128, vt, idesc_o, (n + 15) >> 4,
                                    (cur & kInfoFirst) == 0);
                    if (g == 1 || !(cur & kInfoTwo)) commit(&kv_empty[vat.slot]);
                    if (cur & kInfoLast) commit(&o_full[g]);
                    if (g == 0) nxt = describe();
                    if (ok && nxt && (g == 0 || (nxt & kInfoTwo))) ok = issue_s(nxt, g);
                }
                if (ok && (nxt & kInfoTwo) && !(cur & kInfoTwo)) ok = issue_s(nxt, 1);
                vat.advance(2, p.ring);
                cur = nxt;
            }
            commit(&drain);
            __syncwarp();
            int dummy = 0;
            WaitCtx w2{&dummy, p.dev_status};
            mbar_wait(&drain, 0, w2);
        }
    } else {
        regs_inc<kRegsHigh>();
        // ------------------------------------------------------------ softmax and output of tile g
        const int g = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint32_t ts = tmem + lane_base + kColS + g * 128, to = tmem + lane_base + kColO + g * 128;
        const int ochunks = (p.d + 31) >> 5;
        uint32_t uses = 0, outs = 0;
        int q_at = 0, stored = -1;                  // Q slot of the item's first tile; slot whose output is on its way
        bool ok = true;
        auto release = [&]() {                      // the loader may refill the slot once its output has been read
            if (stored >= 0 && lane == 0) {
                bulk_wait_group_read<0>();
                mbar_arrive(&q_empty[stored]);
            }
            stored = -1;
            __syncwarp();
        };
        // the finished item whose O_g is still in TMEM
        bool pending = false;
        int out_b = 0, out_head = 0, out_q0 = 0, out_slot = 0;
        float inv = 0.0f;
        auto read_out = [&]() {
            if (!warp_wait(&o_full[g], outs & 1u, wc)) return false;
            ++outs;
            tc_fence_after();
            uint8_t* tile = smem + out_slot * tile_bytes;        // its last product is done
            for (int c4 = 0; c4 < ochunks; ++c4) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(to + c4 * 32, o);
                tmem_ld_wait();
                uint8_t* dst = tile + (c4 >> 1) * kChunk + r * 128;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        w[u] = pack_bf16(__uint_as_float(o[8 * i + 2 * u]) * inv, __uint_as_float(o[8 * i + 2 * u + 1]) * inv);
                    *reinterpret_cast<uint4*>(dst + ((((c4 & 1) * 4 + i) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (out_q0 + quarter * 32 < p.Lq)
                    for (int c = 0; c < p.chunks; ++c)
                        tma_store_4d(&tmap_o, tile + c * kChunk + quarter * 32 * 128, c * 64, out_head * p.ao.h,
                                     out_q0 + quarter * 32, out_b * p.ao.b);
                bulk_commit_group();
            }
            stored = out_slot;
            pending = false;
            return true;
        };
        Item item, following = item_of(p, blockIdx.x);      // read ahead by one item
        for (int it = blockIdx.x; ok && it < p.items; it += gridDim.x) {
            item = following;
            if (it + (int)gridDim.x < p.items) following = item_of(p, it + gridDim.x);
            const int slot = (q_at + g) % kQBufs;
            if (item.steps > 0) q_at = (q_at + (item.two ? 2 : 1)) % kQBufs;
            if (g == 1 && !item.two) {
                // nothing to do, but the loader may come to need the tile of the last item this group had
                if (pending && !(ok = read_out())) break;
                release();
                continue;
            }
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < item.steps; ++j, ++uses) {
                if (!warp_wait(&s_full[g], uses & 1u, wc)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int n = min(item.keys - j * kRows, kRows);
                uint32_t v[kRows];
                if (n == kRows) {
#pragma unroll
                    for (int c4 = 0; c4 < 4; ++c4)
                        tmem_ld_32x32b_x32(ts + c4 * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[c4 * 32]));
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int c4 = 0; c4 < 4; ++c4)
                        if (c4 * 32 < n) tmem_ld_32x32b_x32(ts + c4 * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[c4 * 32]));
                    tmem_ld_wait();
                    // keys past the length: -infinity whatever was computed there
#pragma unroll
                    for (int i = 0; i < kRows; ++i)
                        if (i >= n) v[i] = 0xFF800000u;
                }
                float mx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(v[i]);
#pragma unroll
                for (int i = 4; i < kRows; i += 8)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        mx[u] = i + 4 + u < kRows ? max3(mx[u], __uint_as_float(v[i + u]), __uint_as_float(v[i + 4 + u]))
                                                  : fmaxf(mx[u], __uint_as_float(v[i + u]));
                const float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * p.c;
                const bool move = mt > m + 8.0f;
                const float mref = move ? mt : m;
                const float alpha = move ? ex2(m - mt) : 1.0f;     // m = -infinity: 0
                // all logits -infinity so far: P is 0, not NaN
                const float mm = mref == -INFINITY ? 0.0f : -mref;
                F2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
                for (int c2 = 0; c2 < 4; ++c2) {
                    if (c2 * 32 >= n) break;
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        // (all on the hardware's unit: 32768 queries x 512 states, 24 heads of 128, take 214, 214, 231, 246 us
                        // with 0 to 3 of eight pairs on the FMA pipes, two softmax warps per scheduler being bound by instructions)
                        const F2 x = fma2({__uint_as_float(v[c2 * 32 + 2 * i]), __uint_as_float(v[c2 * 32 + 2 * i + 1])}, {p.c, p.c}, {mm, mm});
                        const F2 e = {ex2(x.x), ex2(x.y)};
                        sum[i & 1] = add2(sum[i & 1], e);
                        w[i] = pack_bf16(e.x, e.y);
                    }
                    tmem_st_x16(ts + c2 * 16, w);
                }
                const F2 total = add2(sum[0], sum[1]);
                l = fmaf(l, alpha, total.x + total.y);
                m = mref;
                // O_g rescaled: its previous product is done, for S_g came after it
                if (j >= 1 && __any_sync(0xffffffffu, alpha != 1.0f)) {
                    for (int c4 = 0; c4 < ochunks; ++c4) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(to + c4 * 32, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st_x32(to + c4 * 32, o);
                    }
                }
                if (pending && !(ok = read_out())) break;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[g]);
                if (j == 1 || item.steps == 1) release();
            }
            if (!ok) break;
            int head, q0;
            tile_place(p, item, g, head, q0);
            const int row = q0 + r;
            uint16_t* orow = static_cast<uint16_t*>(p.out.data) + (int64_t)item.b * p.out.batch_stride +
                             (int64_t)row * p.out.token_stride + (int64_t)head * p.out.head_stride;
            if (p.lse && row < p.Lq)
                p.lse[((int64_t)item.b * p.H + head) * p.Lq + row] = item.steps > 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
            if (item.steps == 0) {
                if (row < p.Lq)
                    for (int i = 0; i < p.d; i += 8) *reinterpret_cast<uint4*>(orow + i) = make_uint4(0, 0, 0, 0);
                continue;
            }
            inv = __frcp_rn(l);                     // no logit above -infinity: 0 / 0
            out_b = item.b;
            out_head = head;
            out_q0 = q0;
            out_slot = slot;
            pending = true;
        }
        if (ok && pending) read_out();
        release();
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

cudaError_t launch_forward_tiles(const CrossAttnArgs& a, int num_sms, cudaStream_t stream) {
    FwdParams p{};
    CUtensorMap mq, mk, mv, mo;
    if (a.Lk > 0) {
        if (!make_heads_map(&mq, a.q, a.B, a.Lq, a.H, a.d, kRows, &p.aq) ||
            !make_heads_map(&mk, a.k, a.B, a.Lk, a.Hkv, a.d, kRows, &p.ak) ||
            !make_heads_map(&mv, a.v, a.B, a.Lk, a.Hkv, a.d, kRows, &p.av) ||
            !make_heads_map(&mo, a.out, a.B, a.Lq, a.H, a.d, 32, &p.ao))
            return cudaErrorInvalidValue;
    } else {
        mq = mk = mv = mo = CUtensorMap{};          // no item has keys: nothing is loaded
    }
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
    p.qtiles = (a.Lq + kRows - 1) / kRows;
    p.tiles = p.group * p.qtiles;
    p.pairs = (p.tiles + 1) / 2;
    p.items = a.B * a.Hkv * p.pairs;
    p.chunks = (a.d + 63) / 64;
    const int tile_bytes = p.chunks * kChunk;
    p.ring = (kSmemLimit - 1024 - 1024 - kQBufs * tile_bytes) / tile_bytes;
    if (p.ring > kMaxRing) p.ring = kMaxRing;
    p.dev_status = a.dev_status;
    const int smem = (kQBufs + p.ring) * tile_bytes + 1024;
    // always the same limit: it belongs to the kernel, and another thread may be about to launch with more
    cudaError_t e = cudaFuncSetAttribute(xattn_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit - 2048);
    if (e != cudaSuccess) return e;
    xattn_fwd_kernel<<<p.items < num_sms ? p.items : num_sms, kThreads, smem, stream>>>(mq, mk, mv, mo, p);
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(1);
    return e;
}

}  // namespace xattn

cudaError_t launch_cross_attention(const CrossAttnArgs& a, int num_sms, cudaStream_t stream) {
    // at most 16 rows a key / value head: a tile of 128 would be mostly empty, and its keys in one block's hands
    if ((int64_t)a.H / a.Hkv * a.Lq <= 16) return xattn::launch_forward_few(a, num_sms, stream);
    return xattn::launch_forward_tiles(a, num_sms, stream);
}

}  // namespace nvfp4
