// cache_sm103.cu -- writing a paged key/value cache (fa_cache_append).
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

} // namespace

int append_tokens(int D) { return kAppendThreads / (D / 8); }

cudaError_t launch_append(const AppendParams &p, int blocks, cudaStream_t st)
{
    append_kernel<<<blocks, kAppendThreads, 0, st>>>(p);
    return cudaGetLastError();
}

} // namespace cache
} // namespace fa
