// cache_sm103.cu -- writing a paged key/value cache (fa_cache_append) and shrinking it
// (fa_cache_evict).
#include <atomic>
#include <cstdint>

#include "cache_device.cuh"
#include "cache_internal.h"

namespace fa {
namespace cache {

namespace {

// Row (in rows of the cache) of slot `slot` of (sequence b, KV head h), or -1 where the sequence
// has no such page.
__device__ __forceinline__ long long row_of(const Pages &pg, int Hkv, int b, int h, int slot)
{
    const int at = slot / pg.page;
    if (slot < 0 || at >= pg.max_pages) return -1;
    const int pid = pg.table ? pg.table[(size_t)b * pg.max_pages + at] : b * pg.max_pages + at;
    if (pid < 0 || pid >= pg.num_pages) return -1;
    return ((long long)pid * Hkv + h) * pg.page + (slot - at * pg.page);
}

// ---------------------------------------------------------------- append
// slot n_b + i of every KV head takes the key and value of token path[b, i] (token i without a
// path), i < count[b]; its accumulated weight starts at 0 and its position is start[b] + i.  A copy,
// bound by memory: a thread moves 16 bytes of K and of V, neighbouring threads neighbouring bytes
// of a row.  16384 tokens of 8 KV heads at D = 128 (134 MB read and written) take 22.4 us, 6.0 TB/s;
// the accepted tokens of a step (8 x 24) 2.3 us, which is the launch.
constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p)
{
    grid_wait();
    grid_done_soon();
    const int head = blockIdx.x / p.blocks_per_head, tile = blockIdx.x - head * p.blocks_per_head;
    const int b = head / p.Hkv, h = head - b * p.Hkv;
    const int i = tile * (kAppendThreads / p.chunks) + threadIdx.x / p.chunks, ch = threadIdx.x % p.chunks;
    const int count = p.count ? min(p.count[b], p.T) : p.T;
    if (i >= count) return;
    const int src = p.path ? p.path[(size_t)b * p.T + i] : i;
    if (src < 0 || src >= p.T) return;
    const long long slot = (long long)max(p.seq_len[b], 0) + i;
    if (slot >= p.capacity) return;
    const int start = p.pos ? p.start[b] : 0;
    const long long row = row_of(p.pages, p.Hkv, b, h, (int)slot);
    if (row >= 0) {
        const size_t from = ((size_t)head * p.T + src) * p.chunks + ch, to = (size_t)row * p.chunks + ch;
        const uint4 k = p.k_new[from], v = p.v_new[from];
        p.k[to] = k;
        p.v[to] = v;
    }
    if (ch == 0) {
        const size_t at = (size_t)head * p.capacity + (size_t)slot;
        if (p.weight) p.weight[at] = 0.f;
        if (p.pos) p.pos[at] = start + i;
    }
}

// ---------------------------------------------------------------- eviction
// One cluster of CTAs per (sequence, KV head); CTA r holds the r-th run of the slots.  Each slot gets a
// 32-bit key whose order is the order in which slots are kept: protected positions, then weights
// (NaN above every number, -0 equal to 0).  The last slot that is kept is found by histograms of 11, 11
// and 10 bits of the key, from the top (the cluster's histograms added through distributed shared
// memory); as soon as no more than kCandidates slots match the digits so far, these are ranked against
// each other by key and slot, which is usually after one or two passes.  If all bits have been used, the
// matching slots are equal and the lowest are kept.
//
// Freed slots below `keep` and kept slots at or above it are then listed in order, as many of the one as of
// the other, and the i-th of these moves to the i-th of those: sources and destinations never meet, so the
// rows move in place, in parallel, and no other row is touched.  The lists hold rows, so that a move is two
// dependent round trips: its list entries, then its rows.
//
// Bound by latency: four walks over a CTA's slots (weights, candidates, counts, lists) and 4 cluster barriers (6 where
// a second histogram is needed), most of them followed by a round trip through distributed shared memory; then the
// moves.  Measured, 8 KV heads, D = 128: 8 x 4160 slots to 4096 12.2 us, 4 x 16384 to 2048 34 us (63 MB: 1.8 TB/s); 16
// heads, D = 64, 16 x up to 2000 slots to 777 20.5 us.  Cycles of the phases at 2 GHz, with the clock read between them,
// in first calls of the three cases: weights, positions and first histogram 6300 - 8600, 9900 - 12800, 6000 - 9100;
// histograms added 2900 - 4400, 4300 - 5900, 2200 - 2900; candidates collected and ranked 5000, 11000 - 12600, 3800; moves
// counted 3400, 4200, 2500 and listed 1700, 5600, 3300; last barrier 2900, 1900, 50; moves 3400 - 4100, 25000 - 26600,
// 14300 - 16300.
// kCandidates of 64 to 512 take the same time.
constexpr int kEvictThreads = 512, kEvictWarps = kEvictThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048, kCandidates = 512;
constexpr uint32_t kNoRow = 0xffffffffu;

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_rank()
{
    int r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ int cluster_size()
{
    int r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// The address of *p in the shared memory of CTA `rank` of the cluster, and loads from such addresses.
// A load takes a few hundred nanoseconds: they are issued side by side and used afterwards.
__device__ __forceinline__ uint32_t remote(const void *p, int rank)
{
    uint32_t a = (uint32_t)__cvta_generic_to_shared(p), b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(rank));
    return b;
}
__device__ __forceinline__ int remote_load(uint32_t a)
{
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ unsigned long long remote_load_u64(uint32_t a)
{
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ int4 remote_load4(uint32_t a)
{
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ uint32_t key_of(float w, bool safe)
{
    if (safe) return 0xffffffffu;
    if (w != w) return 0xfffffffeu;
    const uint32_t u = __float_as_uint(w + 0.f);   // -0 becomes 0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kEvictThreads, 2) evict_kernel(const __grid_constant__ EvictParams p)
{
    extern __shared__ uint32_t held[];           // keys, then page numbers
    __shared__ __align__(16) int hist[kBins];
    // the matching slots as key << 32 | ~slot, which is larger for a slot that is kept first: this CTA's, the cluster's
    __shared__ __align__(16) unsigned long long mine[kCandidates], all[kCandidates];
    __shared__ int warp_a[kEvictWarps], warp_b[kEvictWarps];
    __shared__ int cta_a, cta_b, cta_match;
    __shared__ int s_digit, s_need, s_count;
    __shared__ unsigned long long s_last;
    grid_wait();
    grid_done_soon();
    const int C = cluster_size(), rank = cluster_rank();
    const int head = blockIdx.x / C, b = head / p.Hkv, h = head - b * p.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int next_pos = p.last > 0 ? p.next_pos[b] : 0;
    const int n = min(max(p.seq_len[b], 0), p.capacity), m = p.keep;
    const size_t base = (size_t)head * p.capacity;
    if (h == 0 && rank == 0 && tid == 0) p.new_len[b] = min(n, m);
    const bool copy_w = p.weight_out != p.weight, copy_p = p.pos_out != p.pos;
    const int per = (n + C - 1) / C, lo = min(n, rank * per), hi = min(n, lo + per);   // slots of this CTA
    if (n <= m) {   // nothing to evict (the same for the whole cluster)
        for (int s = lo + tid; s < hi; s += kEvictThreads) {
            if (copy_w) p.weight_out[base + s] = p.weight[base + s];
            if (copy_p) p.pos_out[base + s] = p.pos[base + s];
        }
        return;
    }
    auto sync = [&]() {   // of the cluster
        if (C > 1)
            cluster_sync();
        else
            __syncthreads();
    };
    const int from_pos = next_pos - p.last;
    auto key_from = [&](float w, int at) { return key_of(w, at < p.first || (p.last > 0 && at >= from_pos)); };
    auto key = [&](int s) { return s - lo < p.held ? held[s - lo] : key_from(p.weight[base + s], p.pos[base + s]); };
    // page numbers of this CTA's slots, as many as fit
    int *pages = reinterpret_cast<int *>(held + p.held);
    const int page0 = lo / p.pages.page;
    auto row_at = [&](int s) -> uint32_t {
        const int at = s / p.pages.page, i = at - page0;
        int pid;
        if (i < p.paged)
            pid = pages[i];
        else
            pid = p.pages.table ? p.pages.table[(size_t)b * p.pages.max_pages + at] : b * p.pages.max_pages + at;
        if (pid < 0 || pid >= p.pages.num_pages) return kNoRow;
        return ((uint32_t)pid * p.Hkv + h) * p.pages.page + (s - at * p.pages.page);
    };

    for (int i = tid; i < kBins; i += kEvictThreads) hist[i] = 0;
    for (int i = tid; i < p.paged && (page0 + i) * p.pages.page < hi; i += kEvictThreads)
        pages[i] = p.pages.table ? p.pages.table[(size_t)b * p.pages.max_pages + page0 + i] : b * p.pages.max_pages + page0 + i;
    if (tid == 0) cta_match = 0;
    __syncthreads();
    // every slot once: its key, the first histogram (11 bits), and, where the results go elsewhere, a copy of
    // what stays below `keep` (freed slots among them are overwritten by the moves)
#pragma unroll 2
    for (int s = lo + tid; s < hi; s += kEvictThreads) {
        const float w = p.weight[base + s];
        const int at = p.pos[base + s];
        const uint32_t x = key_from(w, at);
        if (s - lo < p.held) held[s - lo] = x;
        atomicAdd(&hist[x >> 21], 1);
        if (s < m) {
            if (copy_w) p.weight_out[base + s] = w;
            if (copy_p) p.pos_out[base + s] = at;
        }
    }

    // ---- the last slot that is kept
    uint32_t prefix = 0;
    int need = m, shift = 32, matches = n;   // slots to be kept among those that match the digits so far
    while (matches > kCandidates && shift > 0) {
        const int bits = shift > 10 ? 11 : 10, below = shift - bits;
        if (shift < 32) {
            sync();   // the histogram of the pass before has been read
            for (int i = tid; i < kBins; i += kEvictThreads) hist[i] = 0;
            __syncthreads();
            for (int s = lo + tid; s < hi; s += kEvictThreads) {
                const uint32_t x = key(s);
                if ((x ^ prefix) >> shift == 0) atomicAdd(&hist[(x >> below) & ((1u << bits) - 1u)], 1);
            }
        }
        sync();
        // thread t: digits kBins - 1 - 4 t down to kBins - 4 - 4 t, added over the cluster
        constexpr int W = 4;
        static_assert(W * kEvictThreads == kBins, "four bins a thread");
        int sum[W] = {0, 0, 0, 0};
        int4 part[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            if (r < C) part[r] = remote_load4(remote(&hist[kBins - W - W * tid], r));
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            if (r < C) {
                sum[0] += part[r].w;
                sum[1] += part[r].z;
                sum[2] += part[r].y;
                sum[3] += part[r].x;
            }
        const int mass = sum[0] + sum[1] + sum[2] + sum[3];
        int upto = mass;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(~0u, upto, d);
            if (lane >= d) upto += x;
        }
        if (lane == 31) warp_a[warp] = upto;
        __syncthreads();
        int above = upto - mass;
        for (int w = 0; w < warp; ++w) above += warp_a[w];
        if (above < need && need <= above + mass) {
            int e = 0;
#pragma unroll
            for (int x = 0; x < W - 1; ++x)
                if (e == x && above + sum[x] < need) {
                    above += sum[x];
                    e = x + 1;
                }
            int count = sum[0];
#pragma unroll
            for (int x = 1; x < W; ++x) count = e == x ? sum[x] : count;
            s_digit = kBins - 1 - W * tid - e;
            s_need = need - above;
            s_count = count;
        }
        __syncthreads();
        prefix |= (uint32_t)s_digit << below;
        need = s_need;
        matches = s_count;
        shift = below;
    }
    // shift > 0 or few matches: rank the matching slots.  Otherwise all of them have the same key.
    const bool ranked = matches <= kCandidates;
    uint32_t last_key = prefix;
    int last_slot = -1;
    if (ranked) {
        for (int s = lo + tid; s < hi; s += kEvictThreads) {
            const uint32_t x = key(s);
            if (shift == 32 || (x ^ prefix) >> shift == 0 || (shift == 0 && x == prefix)) mine[atomicAdd(&cta_match, 1)] = ((unsigned long long)x << 32) | (uint32_t)~s;
        }
        sync();
        const int counts = lane < C ? remote_load(remote(&cta_match, lane)) : 0;   // of CTA `lane`
        int at = 0;
        for (int r = 0; r < C; ++r) {   // warp w copies from CTA w % C on
            const int count = __shfl_sync(~0u, counts, r);
            if (warp % C == r)
                for (int i = (warp / C) * 32 + lane; i < count; i += (kEvictWarps / C) * 32) all[at + i] = remote_load_u64(remote(&mine[i], r));
            at += count;
        }
        __syncthreads();
        // the candidates' ranks, one thread each, two candidates to a read
        if (tid < ((matches + 31) & ~31)) {
            const unsigned long long me = tid < matches ? all[tid] : 0ull;
            int ahead = 0;
#pragma unroll 2
            for (int i = 0; i + 1 < matches; i += 2) {
                const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(&all[i]);
                ahead += (x.x > me) + (x.y > me);
            }
            if (matches & 1) ahead += all[matches - 1] > me;
            if (tid < matches && ahead == need - 1) s_last = me;
        }
        __syncthreads();
        last_key = (uint32_t)(s_last >> 32);
        last_slot = (int)~(uint32_t)s_last;
    }
    // ---- which slots are kept, in the order of the slots: each warp has a run of them
    const int run = (per + kEvictWarps - 1) / kEvictWarps, wlo = min(hi, lo + warp * run), whi = min(hi, wlo + run);
    int before = 0;   // equal slots before this warp's
    if (!ranked) {
        int eq = 0;
        for (int s0 = wlo; s0 < whi; s0 += 32) eq += __popc(__ballot_sync(~0u, s0 + lane < whi && key(s0 + lane) == prefix));
        if (lane == 0) warp_a[warp] = eq;
        __syncthreads();
        if (tid == 0) {
            int x = 0;
            for (int w = 0; w < kEvictWarps; ++w) x += warp_a[w];
            cta_match = x;
        }
        sync();
        const int counts = lane < rank ? remote_load(remote(&cta_match, lane)) : 0;
        before += __reduce_add_sync(~0u, counts);
        for (int w = 0; w < warp; ++w) before += warp_a[w];
        __syncthreads();
    }
    // f(slot, its being one, its being kept)
    auto walk = [&](auto f) {
        int seen = before;
        for (int s0 = wlo; s0 < whi; s0 += 32) {
            const int s = s0 + lane;
            const bool in = s < whi;
            const uint32_t x = in ? key(s) : 0u;
            bool kept;
            if (ranked) {
                kept = in && (x > last_key || (x == last_key && s <= last_slot));
            } else {
                const uint32_t ties = __ballot_sync(~0u, in && x == prefix);
                kept = in && (x > prefix || (x == prefix && seen + __popc(ties & ((1u << lane) - 1u)) < need));
                seen += __popc(ties);
            }
            f(s, in, kept);
        }
    };
    int holes = 0, srcs = 0;
    walk([&](int s, bool in, bool kept) {
        holes += __popc(__ballot_sync(~0u, in && !kept && s < m));
        srcs += __popc(__ballot_sync(~0u, kept && s >= m));
    });
    if (lane == 0) {
        warp_a[warp] = holes;
        warp_b[warp] = srcs;
    }
    __syncthreads();
    if (tid == 0) {
        int x = 0, y = 0;
        for (int w = 0; w < kEvictWarps; ++w) {
            x += warp_a[w];
            y += warp_b[w];
        }
        cta_a = x;
        cta_b = y;
    }
    sync();
    const int far_holes = lane < C ? remote_load(remote(&cta_a, lane)) : 0, far_srcs = lane < C ? remote_load(remote(&cta_b, lane)) : 0;
    const int moved = __reduce_add_sync(~0u, far_holes);
    int hole_at = __reduce_add_sync(~0u, lane < rank ? far_holes : 0), src_at = __reduce_add_sync(~0u, lane < rank ? far_srcs : 0);
    for (int w = 0; w < warp; ++w) {
        hole_at += warp_a[w];
        src_at += warp_b[w];
    }
    uint2 *to = p.to + (size_t)head * p.longest;
    uint2 *from = p.from + (size_t)head * p.longest;
    walk([&](int s, bool in, bool kept) {
        const bool hole = in && !kept && s < m, src = kept && s >= m;
        const uint32_t hb = __ballot_sync(~0u, hole), sb = __ballot_sync(~0u, src);
        const int before_me = (1 << lane) - 1;
        if (hole) to[hole_at + __popc(hb & before_me)] = make_uint2(row_at(s), (uint32_t)s);
        if (src) from[src_at + __popc(sb & before_me)] = make_uint2(row_at(s), (uint32_t)s);
        hole_at += __popc(hb);
        src_at += __popc(sb);
    });
    sync();   // lists written, every weight read, and no CTA leaves while its shared memory is read
    // ---- the moves, all CTAs of the cluster together: a row to `chunks` lanes, four rows at a time
    const int group = kEvictThreads / p.chunks, ch = tid % p.chunks;   // rows that a CTA moves side by side
    const int step = C * group;
    constexpr int U = 4;
    for (int i0 = rank * group + tid / p.chunks; i0 < moved; i0 += U * step) {
        uint2 d[U], s[U];
        uint4 kk[U], vv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            d[u].x = s[u].x = kNoRow;
            if (i0 + u * step < moved) {
                d[u] = to[i0 + u * step];
                s[u] = from[i0 + u * step];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            kk[u] = vv[u] = make_uint4(0, 0, 0, 0);
            if (d[u].x != kNoRow && s[u].x != kNoRow) {
                kk[u] = p.k[(size_t)s[u].x * p.chunks + ch];
                vv[u] = p.v[(size_t)s[u].x * p.chunks + ch];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (d[u].x != kNoRow) {
                p.k[(size_t)d[u].x * p.chunks + ch] = kk[u];
                p.v[(size_t)d[u].x * p.chunks + ch] = vv[u];
            }
            if (ch == 0 && i0 + u * step < moved) p.weight_out[base + d[u].y] = p.weight[base + s[u].y];
            if (ch == 1 && i0 + u * step < moved) p.pos_out[base + d[u].y] = p.pos[base + s[u].y];
        }
    }
}

} // namespace

cudaError_t launch_evict(const EvictParams &p0, cudaStream_t st)
{
    EvictParams p = p0;
    static std::atomic<uint64_t> configured{0};
    static std::atomic<int> sm_count[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    constexpr int kHeldMost = 40960;   // 160 KB of keys
    if (!(configured.load(std::memory_order_acquire) & (1ull << dev))) {
        e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (kHeldMost + 4096) * 4);
        if (e != cudaSuccess) return e;
        int nsm = 0;
        e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        sm_count[dev].store(nsm, std::memory_order_relaxed);
        configured.fetch_or(1ull << dev, std::memory_order_acq_rel);
    }
    // CTAs of a head: one to an SM, with 1024 slots each at least, and a second one to an SM (all clusters run at
    // once) where each would have more than 7168 slots and moves, a move counted as four.  The lengths are not known
    // here, so the capacity stands for them.  With and without the second (us, 8 KV heads, D = 128; slots and moves of
    // a CTA without it): 8 x 4160 -> 4096 slots (2208) 14.3, 12.2; 16 x 4160 -> 4096 (4416) 15.0, 13.4; 4 x 16384 -> 2048
    // (6144) 35.2, 34.4; 8 x 12288 -> 1024 (8192) 29.9, 36.8; 16 x 8192 -> 8000 (8960) 20.9, 24.2; 16 x 5120 -> 4096 (9216)
    // 37.3, 46.0; 8 x 65536 -> 4096 (40960) 110, 165.
    const int heads = p.B * p.Hkv, sms = sm_count[dev].load(std::memory_order_relaxed);
    int C = 1;
    while (C < kMaxCluster && heads * C * 2 <= sms && p.capacity > 1024 * C) C *= 2;
    if (C < kMaxCluster && heads * C * 2 <= 2 * sms && p.capacity + 4ll * p.longest > 7168ll * C) C *= 2;
    const int per = cdiv(p.capacity, C);
    p.held = per < kHeldMost ? per : kHeldMost;
    const int pages = per / p.pages.page + 2;
    p.paged = pages < 4096 ? pages : 4096;
    return launch_overlapped(evict_kernel, dim3((unsigned)(heads * C)), kEvictThreads, (size_t)(p.held + p.paged) * 4, (unsigned)C, st, p);
}

int append_tokens(int D) { return kAppendThreads / (D / 8); }

cudaError_t launch_append(const AppendParams &p, int blocks, cudaStream_t st)
{
    return launch_overlapped(append_kernel, dim3((unsigned)blocks), kAppendThreads, 0, 1, st, p);
}

} // namespace cache
} // namespace fa
