// rotary_sm103.cu -- rotary positions (fa_rotary), and the cache's writes with the rotation on the way (fa_rotary_append).
//
// Pair p of a head turns by position * freq[p]: (a, b) -> amplitude (a cos - b sin, a sin + b cos).  Frequencies are turns in
// 64-bit fixed point, so that position * freq modulo 2^64 is the exact fraction of a turn, at any position, by one integer
// product; its upper 32 bits, as a signed number of half turns, are the argument of sincospif.  (The angle itself in fp32 would be
// off by 0.004 rad at position 65536.)
//
// A thread has 8 pairs of one token (16 elements, two 16-byte chunks) and goes through a run of heads with them, so that sines and
// cosines are computed once for several heads; four heads' loads are in flight at a time.  Neighbouring threads have
// neighbouring chunks, then neighbouring tokens.  Bound by memory.
#include <atomic>
#include <cstdint>

#include <cuda_fp16.h>

#include "cache_device.cuh"
#include "ptx.cuh"
#include "rotary_internal.h"

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

// Pairs (lo, hi) held in matching halves of two words, or in one word each.
template <bool BF16>
__device__ __forceinline__ void turn_words(uint4 &lo, uint4 &hi, bool interleaved, const float *c, const float *s)
{
    uint32_t *x = &lo.x, *y = &hi.x;
    if (interleaved) {   // words of lo hold pairs 0 .. 3, words of hi 4 .. 7
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f = unpack<BF16>(x[i]), g = unpack<BF16>(y[i]);
            turn(f.x, f.y, c[i], s[i]);
            turn(g.x, g.y, c[i + 4], s[i + 4]);
            x[i] = pack2<BF16>(f.x, f.y);
            y[i] = pack2<BF16>(g.x, g.y);
        }
    } else {
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

// PAIRS pairs of a thread: 8, or 1 where rot is not a multiple of 16 (4-byte or 2-byte accesses).
template <bool BF16, int PAIRS, bool APPEND>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Params p)
{
    cache::grid_wait();
    cache::grid_done_soon();
    const int U = p.D / (2 * PAIRS);
    const long long at = (long long)blockIdx.x * kThreads + threadIdx.x, bt = at / U;
    if (bt >= (long long)p.B * p.T) return;
    const int u = (int)(at - bt * U), b = (int)(bt / p.T), t = (int)(bt - (long long)b * p.T);
    int start = 0;
    long long row = -1;   // of the cache, of KV head 0
    long long slot = 0;
    if constexpr (APPEND) {
        if (p.count && t >= p.count[b]) return;
        slot = (long long)max(p.seq_len[b], 0) + t;
        if (!p.start) start = max(p.seq_len[b], 0);
        if (slot < p.capacity) {
            int pid, r;
            cache::page_of(p.pages, b, (int)slot, pid, r);
            if (pid >= 0 && pid < p.pages.num_pages) row = (long long)pid * p.Hkv * p.pages.page + r;
        }
    }
    const int position = p.position ? p.position[bt] : (p.start ? p.start[b] : start) + t;
    // the thread's elements: e0 .. and e1 ..
    const bool mine = u * PAIRS < p.rot / 2;   // rotated ones
    int e0, e1;
    if (!mine || p.interleaved) {
        e0 = u * 2 * PAIRS;
        e1 = e0 + PAIRS;
    } else {
        e0 = u * PAIRS;
        e1 = e0 + p.rot / 2;
    }
    float c[PAIRS], s[PAIRS];
    if (mine) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const uint64_t phase = (uint64_t)(long long)position * p.freq[u * PAIRS + i];
            sincospif((float)(int)(phase >> 32) * 0x1p-31f, &s[i], &c[i]);
            c[i] *= p.amplitude;
            s[i] *= p.amplitude * p.sign;
        }
    }
    const int h0 = blockIdx.y * p.per, h1 = min(h0 + p.per, p.heads);
    if (APPEND && u == 0 && slot < p.capacity) {   // bookkeeping of the keys' heads
        const int k0 = p.heads - 2 * p.Hkv;
        for (int h = max(h0, k0); h < min(h1, k0 + p.Hkv); ++h) {
            const size_t i = ((size_t)b * p.Hkv + (h - k0)) * p.capacity + (size_t)slot;
            if (p.weight) p.weight[i] = 0.f;
            if (p.pos) p.pos[i] = position;
        }
    }
    constexpr int BATCH = 4;
    for (int h = h0; h < h1; h += BATCH) {
        uint4 lo[BATCH], hi[BATCH];
        uint16_t lo1[BATCH], hi1[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (h + i >= h1) break;
            const int n = h + i < p.seg[0].end ? 0 : h + i < p.seg[1].end ? 1 : 2, head = h + i - (n ? p.seg[n - 1].end : 0);
            const Segment &g = p.seg[n];
            const uint16_t *x = static_cast<const uint16_t *>(g.x) + b * g.xb + head * g.xh + t * g.xt;
            if constexpr (PAIRS == 8) {
                lo[i] = *reinterpret_cast<const uint4 *>(x + e0);
                hi[i] = *reinterpret_cast<const uint4 *>(x + e1);
            } else {
                lo1[i] = x[e0];
                hi1[i] = x[e1];
            }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            if (h + i >= h1) break;
            const int n = h + i < p.seg[0].end ? 0 : h + i < p.seg[1].end ? 1 : 2, head = h + i - (n ? p.seg[n - 1].end : 0);
            const Segment &g = p.seg[n];
            if (mine && g.turned) {
                if constexpr (PAIRS == 8) {
                    turn_words<BF16>(lo[i], hi[i], p.interleaved, c, s);
                } else {
                    float2 f = unpack<BF16>((uint32_t)lo1[i] | (uint32_t)hi1[i] << 16);
                    turn(f.x, f.y, c[0], s[0]);
                    const uint32_t w = pack2<BF16>(f.x, f.y);
                    lo1[i] = (uint16_t)w;
                    hi1[i] = (uint16_t)(w >> 16);
                }
            }
            auto store = [&](uint16_t *y) {
                if constexpr (PAIRS == 8) {
                    *reinterpret_cast<uint4 *>(y + e0) = lo[i];
                    *reinterpret_cast<uint4 *>(y + e1) = hi[i];
                } else {
                    y[e0] = lo1[i];
                    y[e1] = hi1[i];
                }
            };
            if (g.y) store(static_cast<uint16_t *>(g.y) + b * g.yb + head * g.yh + t * g.yt);
            if (APPEND && g.pool && row >= 0)
                store(static_cast<uint16_t *>(g.pool == 1 ? p.k : p.v) + ((size_t)row + (size_t)head * p.pages.page) * p.D);
        }
    }
}

template <bool BF16, int PAIRS, bool APPEND>
cudaError_t launch_one(Params p, cudaStream_t st)
{
    const long long threads = (long long)p.B * p.T * (p.D / (2 * PAIRS)), blocks = (threads + kThreads - 1) / kThreads;
    // A thread goes through `per` heads: one where there are few tokens (the smallest call is all latency), more where
    // there are threads enough to fill the card.
    const long long want = (long long)152 * 2048;
    long long per = threads * p.heads / want;
    per = per < 1 ? 1 : per > p.heads ? p.heads : per;
    p.per = (int)per;
    return cache::launch_overlapped(rotary_kernel<BF16, PAIRS, APPEND>, dim3((unsigned)blocks, (unsigned)((p.heads + per - 1) / per)), kThreads, 0, 1, st, p);
}

} // namespace

cudaError_t launch_rotary(const Params &p, bool bf16, bool append, cudaStream_t st)
{
    // 8 pairs a thread where both of its chunks are whole and aligned
    const bool wide = p.rot % 16 == 0;
    if (append) {
        if (wide) return bf16 ? launch_one<true, 8, true>(p, st) : launch_one<false, 8, true>(p, st);
        return bf16 ? launch_one<true, 1, true>(p, st) : launch_one<false, 1, true>(p, st);
    }
    if (wide) return bf16 ? launch_one<true, 8, false>(p, st) : launch_one<false, 8, false>(p, st);
    return bf16 ? launch_one<true, 1, false>(p, st) : launch_one<false, 1, false>(p, st);
}

} // namespace rotary
} // namespace fa
