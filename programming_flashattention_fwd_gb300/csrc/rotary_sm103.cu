// rotary_sm103.cu -- rotary positions (fa_rotary), and the cache's writes with the rotation on the way (fa_rotary_append).
//
// Pair p of a head turns by position * freq[p]: (a, b) -> amplitude (a cos - b sin, a sin + b cos).  Frequencies are turns in
// 64-bit fixed point, so that position * freq modulo 2^64 is the exact fraction of a turn, at any position, by one integer
// product; its upper 32 bits, as a signed number of half turns, are the argument of sincospif.  (The angle itself in fp32 would be
// off by 0.004 rad at position 65536.)  Products and sums are fp32, rounded to the type once; what is not turned is copied.
//
// A thread has 16 elements of a head (two 16-byte chunks, 8 pairs) of one token and goes through a run of heads with them, so that
// sines and cosines are computed once for several heads; three heads' loads are in flight at a time, the first of them
// while the angles are computed.  Neighbouring threads have neighbouring chunks, then neighbouring tokens: where a thread's own two
// chunks lie side by side instead, every 32-byte sector is written in two parts (3 x 1777 tokens of 32 heads at D = 64 11.5 us, 9.3 so).
// Bound by memory.
#include <atomic>
#include <cstdint>

#include <cuda_fp16.h>

#include "cache_device.cuh"
#include "ptx.cuh"
#include "rotary_internal.h"
#include "schedule.h"

namespace fa {
namespace rotary {

namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ float2 unpack(uint32_t x)
{
    if constexpr (BF16) return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}

// (a, b) of one pair turned.
__device__ __forceinline__ void turn(float &a, float &b, float c, float s)
{
    const float x = a, y = b;
    a = fmaf(x, c, -y * s);
    b = fmaf(x, s, y * c);
}

// Pairs (lo, hi) held in matching halves of two words, or, interleaved, in one word each: lo holds four, hi four others.
template <bool BF16>
__device__ __forceinline__ void turn_words(uint4 &lo, uint4 &hi, bool interleaved, bool turn_lo, bool turn_hi, const float *c, const float *s)
{
    uint32_t *x = &lo.x, *y = &hi.x;
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (turn_lo) {
                float2 f = unpack<BF16>(x[i]);
                turn(f.x, f.y, c[i], s[i]);
                x[i] = pack2<BF16>(f.x, f.y);
            }
            if (turn_hi) {
                float2 g = unpack<BF16>(y[i]);
                turn(g.x, g.y, c[i + 4], s[i + 4]);
                y[i] = pack2<BF16>(g.x, g.y);
            }
        }
    } else if (turn_lo) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f = unpack<BF16>(x[i]), g = unpack<BF16>(y[i]);
            turn(f.x, g.x, c[2 * i], s[2 * i]);
            turn(f.y, g.y, c[2 * i + 1], s[2 * i + 1]);
            x[i] = pack2<BF16>(f.x, f.y);
            y[i] = pack2<BF16>(g.x, g.y);
        }
    }
}

// cos and sin of `position` times a frequency, times the amplitude (and the direction).
__device__ __forceinline__ float2 angle(const Params &p, int position, int pair)
{
    const uint64_t phase = (uint64_t)(long long)position * p.freq[pair];
    float s, c;
    sincospif((float)(int)(phase >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c * p.amplitude, s * p.amplitude * p.sign);
}

// What a thread knows of its token (b, t).
struct Token {
    bool here;            // there is such a token, and it counts
    int b, t, position;
    long long slot, row;  // of the cache: the slot, and its row of KV head 0 (-1: none)
};

template <bool APPEND>
__device__ __forceinline__ Token token_at(const Params &p, long long bt)
{
    Token k = {bt < (long long)p.B * p.T, 0, 0, 0, 0, -1};
    if (!k.here) return k;
    k.b = (int)fdiv((uint32_t)bt, p.f_T);   // B T < 2^31
    k.t = (int)bt - k.b * p.T;
    int start = 0;
    if constexpr (APPEND) {
        k.here = !p.count || k.t < p.count[k.b];
        if (!k.here) return k;
        const int n = max(p.seq_len[k.b], 0);
        k.slot = (long long)n + k.t;
        start = n;
        if (k.slot < p.capacity) {
            int pid, r;
            cache::page_of(p.pages, k.b, (int)k.slot, pid, r);
            if (pid >= 0 && pid < p.pages.num_pages) k.row = (long long)pid * p.Hkv * p.pages.page + r;
        }
    }
    k.position = p.position ? p.position[bt] : (p.start ? p.start[k.b] : start) + k.t;
    return k;
}

// Where head h of all segments is read and written.
template <typename T>
__device__ __forceinline__ const Segment &segment_of(const Params &p, const Token &k, int h, const T *&x, T *&y, int &head)
{
    const int n = h < p.seg[0].end ? 0 : h < p.seg[1].end ? 1 : 2;
    const Segment &g = p.seg[n];
    head = h - (n ? p.seg[n - 1].end : 0);
    x = static_cast<const T *>(g.x) + k.b * g.xb + head * g.xh + k.t * g.xt;
    y = g.y ? static_cast<T *>(g.y) + k.b * g.yb + head * g.yh + k.t * g.yt : nullptr;
    return g;
}

// Weight and position of the token's slot of KV heads [from, to).
__device__ __forceinline__ void note(const Params &p, const Token &k, int from, int to)
{
    if (k.slot >= p.capacity) return;
    for (int h = from; h < to; ++h) {
        const size_t i = ((size_t)k.b * p.Hkv + h) * p.capacity + (size_t)k.slot;
        if (p.weight) p.weight[i] = 0.f;
        if (p.pos) p.pos[i] = k.position;
    }
}

// rot a multiple of 16: 8 pairs a thread.
template <bool BF16, bool APPEND>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ Params p)
{
    cache::grid_wait();
    cache::grid_done_soon();
    const int shift = p.D == 64 ? 2 : p.D == 128 ? 3 : 4, half = p.rot / 2;   // log2 of the units of a head
    const int u = threadIdx.x & ((1 << shift) - 1);
    const Token k = token_at<APPEND>(p, ((long long)blockIdx.x * kThreads + threadIdx.x) >> shift);
    if (!k.here) return;
    // The thread's elements: e0 .. e0 + 7 and e1 .. e1 + 7, each beside the next thread's.  Of halves, rotated threads take a pair's two
    // sides, those behind them the two halves of what is not rotated.
    int e0 = u * 8, e1 = e0 + p.D / 2;
    if (!p.interleaved) {
        e1 = e0 + half;
        if (e0 >= half) {
            e0 += half;
            e1 = e0 + p.D / 2 - half;
        }
    }
    const bool turn_lo = e0 < p.rot, turn_hi = e1 < p.rot;   // of halves, both or neither
    constexpr int BATCH = 3;   // (4: 80 registers and 13.5 instead of 12.7 us for 8 x 500 tokens of 48 heads at D = 64)
    const int h0 = blockIdx.y * p.per, h1 = min(h0 + p.per, p.heads);
    uint4 lo[BATCH], hi[BATCH];
    auto load = [&](int first) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (first + i >= h1) break;
            const uint16_t *x;
            uint16_t *y;
            int head;
            segment_of(p, k, first + i, x, y, head);
            lo[i] = *reinterpret_cast<const uint4 *>(x + e0);
            hi[i] = *reinterpret_cast<const uint4 *>(x + e1);
        }
    };
    load(h0);
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i < 4 || !p.interleaved ? turn_lo : turn_hi) {
            const float2 v = angle(p, k.position, p.interleaved ? (i < 4 ? e0 : e1) / 2 + i % 4 : e0 + i);
            c[i] = v.x;
            s[i] = v.y;
        }
    }
    if (APPEND && u == 0) note(p, k, max(h0 - (p.heads - 2 * p.Hkv), 0), min(h1 - (p.heads - 2 * p.Hkv), p.Hkv));
    for (int first = h0; first < h1; first += BATCH) {
        if (first != h0) load(first);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (first + i >= h1) break;
            const uint16_t *x;
            uint16_t *y;
            int head;
            const Segment &g = segment_of(p, k, first + i, x, y, head);
            if (g.turned) turn_words<BF16>(lo[i], hi[i], p.interleaved, turn_lo, turn_hi, c, s);
            auto store = [&](uint16_t *to) {
                *reinterpret_cast<uint4 *>(to + e0) = lo[i];
                *reinterpret_cast<uint4 *>(to + e1) = hi[i];
            };
            if (y) store(y);
            if (APPEND && g.pool && k.row >= 0)
                store(static_cast<uint16_t *>(g.pool == 1 ? p.k : p.v) + ((size_t)k.row + (size_t)head * p.pages.page) * p.D);
        }
    }
}

// Any even rot: a pair a thread, element by element.
template <bool BF16, bool APPEND>
__global__ void __launch_bounds__(kThreads) rotary_pairs_kernel(const __grid_constant__ Params p)
{
    cache::grid_wait();
    cache::grid_done_soon();
    const int U = p.D / 2;
    const long long at = (long long)blockIdx.x * kThreads + threadIdx.x, bt = at / U;
    const Token k = token_at<APPEND>(p, bt);
    if (!k.here) return;
    const int u = (int)(at - bt * U);
    const bool mine = u < p.rot / 2;
    int e0 = 2 * u, e1 = 2 * u + 1;
    if (mine && !p.interleaved) {
        e0 = u;
        e1 = u + p.rot / 2;
    }
    const float2 cs = mine ? angle(p, k.position, u) : make_float2(1.f, 0.f);
    const int h0 = blockIdx.y * p.per, h1 = min(h0 + p.per, p.heads);
    if (APPEND && u == 0) note(p, k, max(h0 - (p.heads - 2 * p.Hkv), 0), min(h1 - (p.heads - 2 * p.Hkv), p.Hkv));
    for (int h = h0; h < h1; ++h) {
        const uint16_t *x;
        uint16_t *y;
        int head;
        const Segment &g = segment_of(p, k, h, x, y, head);
        uint32_t w = (uint32_t)x[e0] | (uint32_t)x[e1] << 16;
        if (mine && g.turned) {
            float2 f = unpack<BF16>(w);
            turn(f.x, f.y, cs.x, cs.y);
            w = pack2<BF16>(f.x, f.y);
        }
        auto store = [&](uint16_t *to) {
            to[e0] = (uint16_t)w;
            to[e1] = (uint16_t)(w >> 16);
        };
        if (y) store(y);
        if (APPEND && g.pool && k.row >= 0)
            store(static_cast<uint16_t *>(g.pool == 1 ? p.k : p.v) + ((size_t)k.row + (size_t)head * p.pages.page) * p.D);
    }
}

// A thread goes through `per` heads: one where even so there are few blocks (the smallest call is all latency: 8 tokens of 40 heads
// 2.3 us, 3.8 with 8 heads a thread), otherwise three at least, which share the angles and are loaded at once (512 tokens of 40
// heads 3.8 us, 5.1 with one), and more where that still leaves 12 blocks an SM.  16384 tokens of 40 heads at D = 128 53 us (6.3 TB/s;
// with values and the cache's writes 76 us, 6.2 TB/s); 3 x 1777 tokens of 32 heads at D = 64, into the rows of a projection, 9.3 us (4.7
// TB/s).  Angles in shared memory, computed once for a block's 8 warps with other heads each: 5 % slower, and 11 instead of 5 us for
// 8 x 2000 tokens of 4 heads.
template <bool BF16, bool APPEND>
cudaError_t launch_one(Params p, cudaStream_t st)
{
    const bool wide = p.rot % 16 == 0;
    const long long threads = (long long)p.B * p.T * (wide ? p.D / 16 : p.D / 2), blocks = (threads + kThreads - 1) / kThreads;
    const long long groups = (12 * 152 + blocks - 1) / blocks;
    long long per = (p.heads + groups - 1) / groups;
    if (per < 3 && blocks * p.heads > 2 * 152) per = 3 < p.heads ? 3 : p.heads;
    p.per = (int)per;
    p.f_T = make_fastdiv((uint32_t)p.T);
    const dim3 grid((unsigned)blocks, (unsigned)((p.heads + per - 1) / per));
    return cache::launch_overlapped(wide ? rotary_kernel<BF16, APPEND> : rotary_pairs_kernel<BF16, APPEND>, grid, kThreads, 0, 1, st, p);
}

} // namespace

cudaError_t launch_rotary(const Params &p, bool bf16, bool append, cudaStream_t st)
{
    if (append) return bf16 ? launch_one<true, true>(p, st) : launch_one<false, true>(p, st);
    return bf16 ? launch_one<true, false>(p, st) : launch_one<false, false>(p, st);
}

} // namespace rotary
} // namespace fa
