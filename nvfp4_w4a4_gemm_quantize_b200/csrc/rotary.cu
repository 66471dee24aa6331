// rotary.cu -- rotary positions with several axes (nvfp4_rotary).
//
// Pair j of a token's head turns by angle[token, j] = position[axis(j)] *
// theta^(-2 i / width(axis)); the angles do not depend on the head.  A block takes
// a few tokens and forms their cos / sin once in shared memory; a thread has one
// place (a 16-byte vector, or one in each half) of one token's heads, reads its
// angles once and turns that place in several heads, all loaded ahead.  (With a
// place per vector and its angles read for each, it was bound by those reads and
// the addresses: 177 instructions a vector, 100 us for 32768 x 24 x 128.)
// The angle is formed in turns (the frequencies come divided by 2 pi, in FP64 from
// the host) and reduced to half a turn in FP64: three FP64 operations per token and
// pair, against 2 H elements moved.
// Bound by memory: every element is read and written once; B200, 32768 x 24 x 128
// bf16: 70 us, 5.8 TB/s, 88 % of the copy rate.
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dit.h"
#include "internal.h"

namespace nvfp4 {
namespace rotary {

constexpr int kThreads = 256;
constexpr int kHeads = 8;                 // heads of a thread (4 with split pairs, two vectors each)

// n / d for 0 <= n < 2^31 as a multiplication (d >= 1): m = ceil(2^(31 + s) / d), 2^s >= d.
struct FastDiv {
    uint32_t d, m, s;                     // used for n < 256 only
};

FastDiv fast_div(uint32_t d) {
    FastDiv f{d, 0, 0};
    while ((1ull << f.s) < d) ++f.s;
    f.m = (uint32_t)(((1ull << (31 + f.s)) + d - 1) / d);
    return f;
}

__device__ __forceinline__ uint32_t divide(uint32_t n, const FastDiv& f) {
    return (uint32_t)(((uint64_t)n * f.m) >> (31 + f.s));
}

struct Params {
    nvfp4_heads x, out;
    const void* positions;
    int64_t pos_batch_stride, pos_token_stride;
    bool pos_f32;
    int L, H, pairs;
    int tokens, tiles;                    // tokens of a block, blocks of a sample
    FastDiv units, splits;                // places of a head; threads that share a token's place, each a part of the heads
    int rotated_units;                    // vectors of a head that hold pairs (split pairs: of each half)
    float sign;                           // -1: turn back
    double turns[kRotaryMaxPairs];        // frequency of a pair, turns per position
    uint8_t axis[kRotaryMaxPairs];
};

template <int BYTES>
struct Word;
template <>
struct Word<16> { typedef uint4 type; };
template <>
struct Word<8> { typedef uint2 type; };
template <>
struct Word<4> { typedef uint32_t type; };
template <>
struct Word<2> { typedef uint16_t type; };

// W values of type T (bf16 as its 16 bits, or FP32) moved as one word.
template <typename T, int W>
union Vec {
    typename Word<sizeof(T) * W>::type word;
    T v[W];
};

__device__ __forceinline__ float to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float to_f32(float f) { return f; }
__device__ __forceinline__ void from_f32(float f, uint16_t& b) { b = __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
__device__ __forceinline__ void from_f32(float f, float& o) { o = f; }

// (u, v) turned; the two products of a sum are rounded as the compiler contracts them.
__device__ __forceinline__ void turn(float& u, float& v, float2 cs) {
    const float a = u * cs.x - v * cs.y, b = u * cs.y + v * cs.x;
    u = a;
    v = b;
}

template <typename T, int W, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads)
rotary_kernel(const __grid_constant__ Params p) {
    constexpr int kAhead = INTERLEAVED ? kHeads : kHeads / 2;
    constexpr int kAngles = INTERLEAVED ? W / 2 : W;         // of a place (W is 1 only with split pairs)
    extern __shared__ float2 cs[];        // [tokens][pairs]
    const int b = blockIdx.x / p.tiles;
    const int l0 = (int)(blockIdx.x - b * p.tiles) * p.tokens;
    const int tokens = min(p.tokens, p.L - l0);
    // this thread's place, token and first head
    const int slot = (int)divide(threadIdx.x, p.units), unit = (int)threadIdx.x - slot * (int)p.units.d;
    const int token = (int)divide((uint32_t)slot, p.splits), head0 = slot - token * (int)p.splits.d;
    const bool live = token < tokens;
    const bool turned = INTERLEAVED || unit < p.rotated_units;
    const int col = turned ? unit * W : p.pairs + unit * W;  // first column
    const T* src = static_cast<const T*>(p.x.data) + (int64_t)b * p.x.batch_stride + (int64_t)(l0 + token) * p.x.token_stride + col;
    T* dst = static_cast<T*>(p.out.data) + (int64_t)b * p.out.batch_stride + (int64_t)(l0 + token) * p.out.token_stride + col;
    const int end = live ? p.H : 0;
    const int step = (int)p.splits.d;

    Vec<T, W> lo[kAhead], hi[INTERLEAVED ? 1 : kAhead];
    auto load = [&](int head) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int h = head + i * step;
            if (h >= end) break;
            const T* from = src + (int64_t)h * p.x.head_stride;
            lo[i].word = *reinterpret_cast<const decltype(lo[i].word)*>(from);
            if (!INTERLEAVED && turned) hi[i].word = *reinterpret_cast<const decltype(hi[i].word)*>(from + p.pairs);
        }
    };
    load(head0);

    for (int i = threadIdx.x; i < tokens * p.pairs; i += kThreads) {
        const int t = i / p.pairs, j = i - t * p.pairs;
        const int64_t at = (int64_t)b * p.pos_batch_stride + (int64_t)(l0 + t) * p.pos_token_stride + p.axis[j];
        const double position = p.pos_f32 ? (double)static_cast<const float*>(p.positions)[at]
                                          : (double)static_cast<const int32_t*>(p.positions)[at];
        const double turns = position * p.turns[j];
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cs[i] = make_float2(c, p.sign * s);
    }
    __syncthreads();

    float2 angle[kAngles];
#pragma unroll
    for (int e = 0; e < kAngles; ++e) {
        const int j = unit * kAngles + e;
        angle[e] = live && j < p.pairs ? cs[token * p.pairs + j] : make_float2(1.0f, 0.0f);
    }
    for (int head = head0; head < end; head += kAhead * step) {
        if (head != head0) load(head);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int h = head + i * step;
            if (h >= end) break;
            T* to = dst + (int64_t)h * p.out.head_stride;
            if (INTERLEAVED) {
#pragma unroll
                for (int e = 0; e < kAngles; ++e) {
                    if (unit * kAngles + e >= p.pairs) break;            // the rest is copied as it is
                    float f = to_f32(lo[i].v[2 * e]), g = to_f32(lo[i].v[2 * e + 1]);
                    turn(f, g, angle[e]);
                    from_f32(f, lo[i].v[2 * e]);
                    from_f32(g, lo[i].v[2 * e + 1]);
                }
            } else if (turned) {
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    float f = to_f32(lo[i].v[e]), g = to_f32(hi[i].v[e]);
                    turn(f, g, angle[e]);
                    from_f32(f, lo[i].v[e]);
                    from_f32(g, hi[i].v[e]);
                }
                *reinterpret_cast<decltype(hi[i].word)*>(to + p.pairs) = hi[i].word;
            }
            *reinterpret_cast<decltype(lo[i].word)*>(to) = lo[i].word;
        }
    }
}

template <typename T, int W, bool INTERLEAVED>
cudaError_t launch(const Params& p, int64_t blocks, cudaStream_t stream) {
    rotary_kernel<T, W, INTERLEAVED><<<(unsigned)blocks, kThreads, (size_t)p.tokens * p.pairs * sizeof(float2), stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(1);
    return e;
}

// The widest vector (at most 16 bytes) that divides `a` and `b` values.
int vector_values(int64_t a, int64_t b, int most) {
    int w = most;
    while (w > 1 && (a % w != 0 || b % w != 0)) w /= 2;
    return w;
}

}  // namespace rotary

cudaError_t launch_rotary(const RotaryArgs& a, int num_sms, cudaStream_t stream) {
    using namespace rotary;
    Params p{};
    p.x = a.x;
    p.out = a.out;
    p.positions = a.positions;
    p.pos_batch_stride = a.pos_batch_stride;
    p.pos_token_stride = a.pos_token_stride;
    p.pos_f32 = a.pos_f32;
    p.L = (int)a.L;
    p.H = (int)a.H;
    p.pairs = a.pairs;
    p.sign = a.inverse ? -1.0f : 1.0f;
    // theta^(-k / n) as a product of two powers, so that 32 pairs take 11 calls instead of 32 (64-bit: two roundings more)
    int j = 0;
    for (int i = 0; i < a.n_axes; ++i) {
        const int n = a.axis_pairs[i];
        double low[8], high = 1.0;
        for (int k = 0; k < n; ++k, ++j) {
            if (k < 8) low[k] = std::pow(a.theta, -(double)k / n) / 6.283185307179586476925287;
            if (k % 8 == 0) high = k == 0 ? 1.0 : std::pow(a.theta, -(double)k / n);
            p.turns[j] = low[k % 8] * high;
            p.axis[j] = (uint8_t)i;
        }
    }
    const int most = a.f32 ? 4 : 8;
    // interleaved pairs: d % 8 == 0, so full vectors; split pairs: a vector
    // must not straddle the halves or the copied tail
    const int w = a.interleaved ? most : vector_values(a.pairs, a.d - 2 * a.pairs, most);
    const int units = a.interleaved ? (int)a.d / w : (a.pairs + (int)(a.d - 2 * a.pairs)) / w;
    p.rotated_units = a.interleaved ? units : a.pairs / w;
    // threads that share a token's place: as many as leave each a batch of heads, more (fewer heads, fewer tokens of a
    // block) while the blocks would not fill the SMs twice
    const int slots = kThreads / units;
    int heads = a.interleaved ? kHeads : kHeads / 2;
    int64_t tokens = 1;
    int splits = 1;
    while (true) {
        splits = (int)((a.H + heads - 1) / heads);
        if (splits > slots) splits = slots;
        tokens = slots / splits;
        if (heads == 1 || a.B * ((a.L + tokens - 1) / tokens) >= 2 * num_sms) break;
        heads = (heads + 1) / 2;
    }
    if (tokens > a.L) tokens = a.L;
    p.units = fast_div((uint32_t)units);
    p.splits = fast_div((uint32_t)splits);
    p.tokens = (int)tokens;
    p.tiles = (int)((a.L + tokens - 1) / tokens);
    const int64_t blocks = a.B * p.tiles;
    if (a.f32) {
        if (a.interleaved) return launch<float, 4, true>(p, blocks, stream);
        if (w == 4) return launch<float, 4, false>(p, blocks, stream);
        if (w == 2) return launch<float, 2, false>(p, blocks, stream);
        return launch<float, 1, false>(p, blocks, stream);
    }
    if (a.interleaved) return launch<uint16_t, 8, true>(p, blocks, stream);
    if (w == 8) return launch<uint16_t, 8, false>(p, blocks, stream);
    if (w == 4) return launch<uint16_t, 4, false>(p, blocks, stream);
    if (w == 2) return launch<uint16_t, 2, false>(p, blocks, stream);
    return launch<uint16_t, 1, false>(p, blocks, stream);
}

}  // namespace nvfp4
