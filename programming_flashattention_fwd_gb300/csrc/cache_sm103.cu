// cache_sm103.cu -- writing a paged key/value cache (fa_cache_append) and shrinking it
// (fa_cache_evict).
#include <atomic>
#include <cstdint>

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
    const int pid = pg.table ? __ldg(pg.table + (size_t)b * pg.max_pages + at) : b * pg.max_pages + at;
    if (pid < 0 || pid >= pg.num_pages) return -1;
    return ((long long)pid * Hkv + h) * pg.page + (slot - at * pg.page);
}

// ---------------------------------------------------------------- append
// slot n_b + i of every KV head takes the key and value of token path[b, i] (token i without a
// path), i < count[b]; its accumulated weight starts at 0 and its position is start[b] + i.  A copy,
// bound by memory: a thread moves 16 bytes of K and of V, neighbouring threads neighbouring bytes
// of a row.
constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p)
{
    const int head = blockIdx.x / p.blocks_per_head, tile = blockIdx.x - head * p.blocks_per_head;
    const int b = head / p.Hkv, h = head - b * p.Hkv;
    const int i = tile * (kAppendThreads / p.chunks) + threadIdx.x / p.chunks, ch = threadIdx.x % p.chunks;
    const int count = p.count ? min(__ldg(p.count + b), p.T) : p.T;
    if (i >= count) return;
    const int src = p.path ? __ldg(p.path + (size_t)b * p.T + i) : i;
    if (src < 0 || src >= p.T) return;
    const long long slot = (long long)max(__ldg(p.seq_len + b), 0) + i;
    if (slot >= p.capacity) return;
    const long long row = row_of(p.pages, p.Hkv, b, h, (int)slot);
    if (row >= 0) {
        const size_t from = ((size_t)head * p.T + src) * p.chunks + ch, to = (size_t)row * p.chunks + ch;
        const uint4 k = __ldg(p.k_new + from), v = __ldg(p.v_new + from);
        p.k[to] = k;
        p.v[to] = v;
    }
    if (ch == 0) {
        const size_t at = (size_t)head * p.capacity + (size_t)slot;
        if (p.weight) p.weight[at] = 0.f;
        if (p.pos) p.pos[at] = __ldg(p.start + b) + i;
    }
}

// ---------------------------------------------------------------- eviction
// One cluster of CTAs per (sequence, KV head); CTA r holds the r-th run of the slots.  Each slot gets a
// 32-bit key whose order is the order in which slots are kept: protected positions, then weights
// (NaN above every number, -0 equal to 0).  The key of the last slot that is kept is found digit by
// digit (8 bits a pass, the cluster's histograms added through distributed shared memory); of the
// slots with just that key the lowest are kept.  Freed slots below `keep` and kept slots at or above it
// are then listed in order, as many of the one as of the other, and the i-th of these moves to the i-th of
// those: sources and destinations never meet, so the rows move in place, in parallel, and no other
// row is touched.
constexpr int kEvictThreads = 512, kEvictWarps = kEvictThreads / 32;
constexpr int kMaxCluster = 8;

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
// *p in the shared memory of CTA `rank` of the cluster
__device__ __forceinline__ int remote(const int *p, int rank)
{
    uint32_t a = (uint32_t)__cvta_generic_to_shared(p), b;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(b) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t key_of(float w, bool safe)
{
    if (safe) return 0xffffffffu;
    if (w != w) return 0xfffffffeu;
    const uint32_t u = __float_as_uint(w + 0.f);   // -0 becomes 0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const __grid_constant__ EvictParams p)
{
    extern __shared__ uint32_t held[];
    __shared__ int hist[4][256];
    __shared__ int total[256];
    __shared__ int warp_eq[kEvictWarps], warp_hole[kEvictWarps], warp_src[kEvictWarps];
    __shared__ int cta_hole, cta_src;
    __shared__ uint32_t s_digit;
    __shared__ int s_need;
    const int C = cluster_size(), rank = cluster_rank();
    const int head = blockIdx.x / C, b = head / p.Hkv, h = head - b * p.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = min(max(__ldg(p.seq_len + b), 0), p.capacity), m = p.keep;
    const int left = min(n, m);
    const size_t base = (size_t)head * p.capacity;
    if (h == 0 && rank == 0 && tid == 0) p.new_len[b] = left;
    const bool copy_w = p.weight_out != p.weight, copy_p = p.pos_out != p.pos;
    // slots of this CTA, and of each of its warps: consecutive runs
    const int per = (n + C - 1) / C, lo = min(n, rank * per), hi = min(n, lo + per);
    if (n <= m) {   // nothing to evict (the same for the whole cluster)
        for (int s = lo + tid; s < hi; s += kEvictThreads) {
            if (copy_w) p.weight_out[base + s] = p.weight[base + s];
            if (copy_p) p.pos_out[base + s] = p.pos[base + s];
        }
        return;
    }
    const int from = p.last > 0 ? __ldg(p.next_pos + b) - p.last : 0x7fffffff;
    auto key_from_memory = [&](int s) {
        const int at = p.pos[base + s];
        return key_of(p.weight[base + s], at < p.first || (p.last > 0 && at >= from));
    };
    auto key = [&](int s) { return s - lo < p.held ? held[s - lo] : key_from_memory(s); };

    for (int i = tid; i < 4 * 256; i += kEvictThreads) (&hist[0][0])[i] = 0;
    for (int s = lo + tid; s < min(hi, lo + p.held); s += kEvictThreads) held[s - lo] = key_from_memory(s);
    __syncthreads();

    // ---- the key of the last slot that is kept, from its highest digit down
    uint32_t prefix = 0;
    int need = m;            // slots still to be found among those that match the digits so far
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        for (int s0 = lo; s0 < hi; s0 += kEvictThreads) {
            const int s = s0 + tid;
            uint32_t digit = 256;
            if (s < hi) {
                const uint32_t x = key(s);
                if (pass == 0 || (x ^ prefix) >> (shift + 8) == 0) digit = (x >> shift) & 255u;
            }
            const uint32_t same = __match_any_sync(~0u, digit);
            if (digit < 256 && lane == __ffs(same) - 1) atomicAdd(&hist[pass][digit], __popc(same));
        }
        cluster_sync();
        if (tid < 256) {
            int x = 0;
            for (int r = 0; r < C; ++r) x += remote(&hist[pass][tid], r);
            total[tid] = x;
        }
        __syncthreads();
        if (warp == 0) {   // lane l: digits 255 - 8 l down to 248 - 8 l
            int mine = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) mine += total[255 - 8 * lane - e];
            int upto = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int x = __shfl_up_sync(~0u, upto, d);
                if (lane >= d) upto += x;
            }
            const uint32_t reach = __ballot_sync(~0u, upto >= need);
            if (lane == __ffs(reach) - 1) {
                int above = upto - mine, d = 255 - 8 * lane;
                while (above + total[d] < need) above += total[d--];
                s_digit = (uint32_t)d;
                s_need = need - above;
            }
        }
        __syncthreads();
        prefix |= s_digit << shift;
        need = s_need;
    }
    // ---- of the slots with this very key, the first `need` are kept: those before this CTA and warp
    int before = 0;
    for (int r = 0; r < rank; ++r) before += remote(&hist[3][prefix & 255u], r);
    const int run = (per + kEvictWarps - 1) / kEvictWarps, wlo = min(hi, lo + warp * run), whi = min(hi, wlo + run);
    int eq = 0;
    for (int s0 = wlo; s0 < whi; s0 += 32) eq += __popc(__ballot_sync(~0u, s0 + lane < whi && key(s0 + lane) == prefix));
    if (lane == 0) warp_eq[warp] = eq;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += warp_eq[w];
    // walks this warp's slots in order: f(slot, kept)
    auto walk = [&](auto f) {
        int seen = before;
        for (int s0 = wlo; s0 < whi; s0 += 32) {
            const int s = s0 + lane;
            const uint32_t x = s < whi ? key(s) : 0u;
            const bool tie = s < whi && x == prefix;
            const uint32_t ties = __ballot_sync(~0u, tie);
            const bool kept = s < whi && (x > prefix || (tie && seen + __popc(ties & ((1u << lane) - 1u)) < need));
            seen += __popc(ties);
            f(s, s < whi, kept);
        }
    };
    int holes = 0, srcs = 0;
    walk([&](int s, bool in, bool kept) {
        holes += __popc(__ballot_sync(~0u, in && !kept && s < m));
        srcs += __popc(__ballot_sync(~0u, kept && s >= m));
    });
    if (lane == 0) {
        warp_hole[warp] = holes;
        warp_src[warp] = srcs;
    }
    __syncthreads();
    if (tid == 0) {
        int a = 0, c = 0;
        for (int w = 0; w < kEvictWarps; ++w) {
            a += warp_hole[w];
            c += warp_src[w];
        }
        cta_hole = a;
        cta_src = c;
    }
    cluster_sync();
    int hole_at = 0, src_at = 0, moved = 0;
    for (int r = 0; r < C; ++r) {
        const int a = remote(&cta_hole, r), c = remote(&cta_src, r);
        if (r < rank) {
            hole_at += a;
            src_at += c;
        }
        moved += a;
    }
    for (int w = 0; w < warp; ++w) {
        hole_at += warp_hole[w];
        src_at += warp_src[w];
    }
    int32_t *dst_of = p.moves + (size_t)head * 2 * p.longest, *src_of = dst_of + p.longest;
    walk([&](int s, bool in, bool kept) {
        const bool hole = in && !kept && s < m, src = kept && s >= m;
        const uint32_t hb = __ballot_sync(~0u, hole), sb = __ballot_sync(~0u, src);
        if (hole) dst_of[hole_at + __popc(hb & ((1u << lane) - 1u))] = s;
        if (src) src_of[src_at + __popc(sb & ((1u << lane) - 1u))] = s;
        hole_at += __popc(hb);
        src_at += __popc(sb);
        if (kept && s < m) {
            if (copy_w) p.weight_out[base + s] = p.weight[base + s];
            if (copy_p) p.pos_out[base + s] = p.pos[base + s];
        }
    });
    cluster_sync();   // lists written, every key read, and no CTA leaves while its histograms are read
    // ---- the moves, all CTAs of the cluster together
    for (int x = rank * kEvictThreads + tid; x < moved * p.chunks; x += C * kEvictThreads) {
        const int i = x / p.chunks, ch = x - i * p.chunks;
        const int s = src_of[i], d = dst_of[i];
        const long long rs = row_of(p.pages, p.Hkv, b, h, s), rd = row_of(p.pages, p.Hkv, b, h, d);
        if (rd >= 0) {
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const uint4 a = rs >= 0 ? p.k[(size_t)rs * p.chunks + ch] : zero, c = rs >= 0 ? p.v[(size_t)rs * p.chunks + ch] : zero;
            p.k[(size_t)rd * p.chunks + ch] = a;
            p.v[(size_t)rd * p.chunks + ch] = c;
        }
        if (ch == 0) {
            p.weight_out[base + d] = p.weight[base + s];
            p.pos_out[base + d] = p.pos[base + s];
        }
    }
}

} // namespace

cudaError_t launch_evict(const EvictParams &p0, cudaStream_t st)
{
    EvictParams p = p0;
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    constexpr int kHeldMost = 40960;   // 160 KB of keys
    if (!(configured.load(std::memory_order_acquire) & (1ull << dev))) {
        e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldMost * 4);
        if (e != cudaSuccess) return e;
        configured.fetch_or(1ull << dev, std::memory_order_acq_rel);
    }
    // CTAs of a head: enough for about two in each SM, but with 1024 slots each at least
    const int heads = p.B * p.Hkv;
    int C = 1;
    while (C < kMaxCluster && heads * C * 2 <= 304 && p.capacity > 1024 * C) C *= 2;
    const int per = cdiv(p.capacity, C);
    p.held = per < kHeldMost ? per : kHeldMost;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(heads * C));
    cfg.blockDim = dim3(kEvictThreads);
    cfg.dynamicSmemBytes = (size_t)p.held * 4;
    cfg.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)C;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_kernel, p);
}

int append_tokens(int D) { return kAppendThreads / (D / 8); }

cudaError_t launch_append(const AppendParams &p, int blocks, cudaStream_t st)
{
    append_kernel<<<blocks, kAppendThreads, 0, st>>>(p);
    return cudaGetLastError();
}

} // namespace cache
} // namespace fa
