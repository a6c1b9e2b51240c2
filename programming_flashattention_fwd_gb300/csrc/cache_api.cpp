// cache_api.cpp -- the cache operators of include/fa.h: argument checks (before any CUDA call),
// tensor maps and dispatch to the kernels.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "cache_internal.h"
#include "fa.h"
#include "fa_internal.h"

namespace {

using namespace fa::cache;
using EncodeTiledFn = PFN_cuTensorMapEncodeTiled_v12000;

EncodeTiledFn encode_fn()
{
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

// A dense row-major 16-bit tensor, innermost extent first; boxes of 64 columns x `rows` rows x 1,
// 128-byte swizzle.
bool encode(CUtensorMap *m, const void *base, bool bf16, int rank, const long long *extent, int rows)
{
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[4], strides[3], pitch = 2;
    cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, estr[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        dims[i] = (cuuint64_t)extent[i];
        pitch *= dims[i];
        if (i + 1 < rank) strides[i] = pitch;
    }
    return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank,
               const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Range {
    uintptr_t at;
    size_t bytes;
};

Range range(const void *p, size_t bytes) { return Range{reinterpret_cast<uintptr_t>(p), p ? bytes : 0}; }
bool overlap(Range a, Range b) { return a.bytes && b.bytes && a.at < b.at + b.bytes && b.at < a.at + a.bytes; }

// Whether a written range meets any other of `all` (n ranges, the first `written` of them written).
bool clash(const Range *all, int n, int written)
{
    for (int i = 0; i < written; ++i)
        for (int j = 0; j < n; ++j)
            if (i != j && overlap(all[i], all[j])) return true;
    return false;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Positive and finite, with its factor log2 e too.
bool good_scale(float s) { return s > 0.f && std::isfinite((float)((double)s * 1.4426950408889634)); }

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// Checks of a cache's own fields, shared by every entry point.
int check_cache(const fa_cache_t *c)
{
    if (!c) return FA_ERR_NULL_PTR;
    if (c->dtype != 0 && c->dtype != 1) return FA_ERR_ARG;
    if (c->B < 0 || c->max_pages < 0 || c->num_pages < 0) return FA_ERR_BAD_DIM;
    if (c->Hkv < 1) return FA_ERR_HEADS;
    if (c->D != 64 && c->D != 128 && c->D != 256) return FA_ERR_UNSUPPORTED_D;
    if (c->page < 16 || c->page % 16 != 0) return FA_ERR_BAD_DIM;
    const long long cap = (long long)c->max_pages * c->page;
    // the kernels' loops step over a sequence's end by up to 512 slots, in 32 bits
    if (cap > 0x7fffffffLL - 1024 || (long long)c->B * c->Hkv > 0x7fffffffLL || (long long)c->B * c->max_pages > 0x7fffffffLL)
        return FA_ERR_BAD_DIM;
    // slots without any page to be in; a dense cache without pages enough
    if ((c->num_pages == 0 && cap > 0) || (!c->table && (long long)c->B * c->max_pages > c->num_pages)) return FA_ERR_BAD_DIM;
    return FA_OK;
}

// The pointers of a non-empty cache.
int check_cache_pointers(const fa_cache_t *c)
{
    if (!c->seq_len || (c->num_pages > 0 && (!c->k || !c->v))) return FA_ERR_NULL_PTR;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->table, 4) || !aligned(c->seq_len, 4)) return FA_ERR_ALIGN;
    return FA_OK;
}

size_t pool_bytes(const fa_cache_t *c) { return (size_t)c->num_pages * c->Hkv * c->page * c->D * 2; }

Pages pages_of(const fa_cache_t *c) { return Pages{c->table, c->page, c->max_pages, c->num_pages}; }

// K or V of a cache as a (D, page, Hkv, num_pages) tensor.  An empty pool (the capacity is 0 then, so no length
// makes a kernel read it) is given one page of extent so that the map can be encoded over any valid address.
bool encode_pool(CUtensorMap *m, const void *base, const void *any, const fa_cache_t *c, int rows)
{
    const long long ext[4] = {c->D, c->page, c->Hkv, c->num_pages > 0 ? c->num_pages : 1};
    return encode(m, c->num_pages > 0 ? base : any, c->dtype == 0, 4, ext, rows);
}

} // namespace

extern "C" {

size_t fa_tree_workspace_bytes(int Hq, int Hkv, int T, int D)
{
    if (Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || T < 1 || D < 1) return 0;
    const long long rows = (long long)(Hq / Hkv) * T, tile = tree_tile(D, rows);
    const size_t part = (size_t)(rows < tile ? rows : tile);
    return (size_t)kMaxCtas * sizeof(Cut) + (size_t)2 * kMaxCtas * part * (D + 1) * 4;
}

int fa_tree_debug(const fa_cache_t *cache, const void *q, const void *k_new, const void *v_new, const int32_t *parent,
                  const int32_t *draft_len, void *o, float *lse, int Hq, int T, float scale, void *workspace,
                  size_t workspace_bytes, fa_stream_t stream, uint64_t timeout_ns, uint32_t inject)
{
    int st = check_cache(cache);
    if (st != FA_OK) return st;
    const int B = cache->B, Hkv = cache->Hkv, D = cache->D;
    if (T < 0) return FA_ERR_BAD_DIM;
    if (Hq < 1 || Hq % Hkv != 0) return FA_ERR_HEADS;
    if (!good_scale(scale)) return FA_ERR_SCALE;
    if (B == 0 || T == 0) return FA_OK;
    const long long rows = (long long)(Hq / Hkv) * T;
    const int tile = tree_tile(D, rows), BN = 1 << tree_log_keys(D), cap = cache->max_pages * cache->page;
    const long long mt = (rows + tile - 1) / tile;
    const long long steps = ((long long)cap + BN - 1) / BN + (T + BN - 1) / BN;
    if (rows > 0x7fffffffLL - 256 || (double)B * Hkv * mt * steps > 2147483647.0) return FA_ERR_BAD_DIM;
    st = check_cache_pointers(cache);
    if (st != FA_OK) return st;
    if (!q || !k_new || !v_new || !o || !lse || !workspace) return FA_ERR_NULL_PTR;
    if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
        !aligned(parent, 4) || !aligned(draft_len, 4) || !aligned(workspace, 32))
        return FA_ERR_ALIGN;
    const size_t need = fa_tree_workspace_bytes(Hq, Hkv, T, D);
    if (workspace_bytes < need) return FA_ERR_TOO_LARGE;
    const size_t nq = (size_t)B * Hq * T * D * 2, nn = (size_t)B * Hkv * T * D * 2;
    const Range all[] = {range(o, nq), range(lse, (size_t)B * Hq * T * 4), range(workspace, need), range(q, nq), range(k_new, nn),
                         range(v_new, nn), range(cache->k, pool_bytes(cache)), range(cache->v, pool_bytes(cache)),
                         range(cache->table, (size_t)B * cache->max_pages * 4), range(cache->seq_len, (size_t)B * 4),
                         range(parent, (size_t)B * T * 4), range(draft_len, (size_t)B * 4)};
    if (clash(all, sizeof(all) / sizeof(all[0]), 3)) return FA_ERR_ALIAS;
    st = fa::check_device();
    if (st != FA_OK) return st;

    const bool bf16 = cache->dtype == 0;
    const int box = gcd(cache->page, 128) < BN ? gcd(cache->page, 128) : BN;
    TreeMaps m;
    std::memset(&m, 0, sizeof(m));
    const long long eq[3] = {D, rows, (long long)B * Hkv}, en[3] = {D, T, (long long)B * Hkv};
    // a tile of up to 64 rows leaves the other rows of its 128-row operand to whatever is behind it (no one
    // reads what becomes of them), so that two query tiles fit where one of 128 rows does
    const bool small = rows <= 64;
    const int q_rows = small ? (int)((rows + 7) / 8 * 8) : kRowTile;
    if (!encode(&m.q, q, bf16, 3, eq, q_rows) || !encode(&m.k_new, k_new, bf16, 3, en, BN) ||
        !encode(&m.v_new, v_new, bf16, 3, en, BN) || !encode_pool(&m.k, cache->k, q, cache, box) ||
        !encode_pool(&m.v, cache->v, q, cache, box))
        return FA_ERR_TENSORMAP;

    TreeParams p;
    std::memset(&p, 0, sizeof(p));
    p.s = TreeShape{B, Hkv, T, (int)rows, tile, (int)mt, tree_log_keys(D), cap, cache->seq_len, draft_len};
    p.pages = pages_of(cache);
    p.parent = parent;
    p.v_new = v_new;
    p.o = o;
    p.lse = lse;
    p.part_rows = rows < tile ? (int)rows : tile;
    p.q_panel = small ? 8192 : 16384;
    p.q_bufs = small ? 2 : 1;
    p.q_box = q_rows * 128;
    p.cuts = static_cast<Cut *>(workspace);
    p.part_o = reinterpret_cast<float *>(p.cuts + kMaxCtas);   // a multiple of 32 bytes on
    p.part_lse = p.part_o + (size_t)2 * kMaxCtas * p.part_rows * D;
    p.box_rows = box;
    p.sl2 = (float)((double)scale * 1.4426950408889634);
    p.timeout_ns = timeout_ns;
    p.inject = inject;
    return launch_tree(D, bf16, m, p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

int fa_tree_fwd(const fa_cache_t *cache, const void *q, const void *k_new, const void *v_new, const int32_t *parent,
                const int32_t *draft_len, void *o, float *lse, int Hq, int T, float scale, void *workspace,
                size_t workspace_bytes, fa_stream_t stream)
{
    return fa_tree_debug(cache, q, k_new, v_new, parent, draft_len, o, lse, Hq, T, scale, workspace, workspace_bytes, stream, 0, 0);
}

int fa_cache_append(const fa_cache_t *cache, const void *k_new, const void *v_new, const int32_t *path, const int32_t *count,
                    const int32_t *start, float *weight, int32_t *pos, int T, fa_stream_t stream)
{
    int st = check_cache(cache);
    if (st != FA_OK) return st;
    const int B = cache->B, Hkv = cache->Hkv, D = cache->D;
    if (T < 0) return FA_ERR_BAD_DIM;
    if (B == 0 || T == 0) return FA_OK;
    st = check_cache_pointers(cache);
    if (st != FA_OK) return st;
    if (!k_new || !v_new || (path && !count) || (pos && !start)) return FA_ERR_NULL_PTR;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(path, 4) || !aligned(count, 4) || !aligned(start, 4) ||
        !aligned(weight, 4) || !aligned(pos, 4))
        return FA_ERR_ALIGN;
    const int cap = cache->max_pages * cache->page, per = append_tokens(D);
    const long long tiles = ((long long)T + per - 1) / per, blocks = (long long)B * Hkv * tiles;
    if (blocks > 0x7fffffffLL) return FA_ERR_BAD_DIM;
    const size_t nn = (size_t)B * Hkv * T * D * 2, ns = (size_t)B * Hkv * cap * 4;
    const Range all[] = {range(cache->k, pool_bytes(cache)), range(cache->v, pool_bytes(cache)), range(weight, ns), range(pos, ns),
                         range(k_new, nn), range(v_new, nn), range(cache->table, (size_t)B * cache->max_pages * 4),
                         range(cache->seq_len, (size_t)B * 4), range(path, (size_t)B * T * 4), range(count, (size_t)B * 4),
                         range(start, (size_t)B * 4)};
    if (clash(all, sizeof(all) / sizeof(all[0]), 4)) return FA_ERR_ALIAS;
    st = fa::check_device();
    if (st != FA_OK) return st;
    AppendParams p;
    std::memset(&p, 0, sizeof(p));
    p.pages = pages_of(cache);
    p.k = static_cast<uint4 *>(cache->k);
    p.v = static_cast<uint4 *>(cache->v);
    p.k_new = static_cast<const uint4 *>(k_new);
    p.v_new = static_cast<const uint4 *>(v_new);
    p.seq_len = cache->seq_len;
    p.path = path;
    p.count = count;
    p.start = start;
    p.weight = weight;
    p.pos = pos;
    p.B = B;
    p.Hkv = Hkv;
    p.T = T;
    p.capacity = cap;
    p.chunks = D / 8;
    p.blocks_per_head = (int)tiles;
    return launch_append(p, (int)blocks, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

size_t fa_weights_workspace_bytes(void) { return (size_t)kMaxCtas * sizeof(Cut) + (size_t)2 * kMaxCtas * 256 * 4; }

int fa_weights_debug(const fa_cache_t *cache, const void *q, const float *lse, const int32_t *path, const int32_t *count,
                     const float *weight, float *out, int Hq, int T, int causal, float scale, void *workspace,
                     size_t workspace_bytes, fa_stream_t stream, uint64_t timeout_ns, uint32_t inject)
{
    int st = check_cache(cache);
    if (st != FA_OK) return st;
    const int B = cache->B, Hkv = cache->Hkv, D = cache->D;
    if (T < 0) return FA_ERR_BAD_DIM;
    if (Hq < 1 || Hq % Hkv != 0) return FA_ERR_HEADS;
    if (!good_scale(scale)) return FA_ERR_SCALE;
    if (causal != 0 && causal != 1) return FA_ERR_CAUSAL;
    const int group = Hq / Hkv, NQ = weigh_rows(D), cap = cache->max_pages * cache->page;
    if (B == 0 || cap == 0) return FA_OK;
    if (T == 0) return FA_ERR_BAD_DIM;
    const long long rows = (long long)group * T, kt = ((long long)cap + 127) / 128;
    if (rows > 0x7fffffffLL - 128 || (double)B * Hq > 2147483647.0 ||
        (double)B * Hkv * kt * ((double)group * ((T + NQ - 1) / NQ) + 1) > 2147483647.0)
        return FA_ERR_BAD_DIM;
    st = check_cache_pointers(cache);
    if (st != FA_OK) return st;
    if (!q || !lse || !out || !workspace || (path && !count)) return FA_ERR_NULL_PTR;
    if (!aligned(q, 16) || !aligned(lse, 4) || !aligned(path, 4) || !aligned(count, 4) || !aligned(weight, 4) || !aligned(out, 4) ||
        !aligned(workspace, 16))
        return FA_ERR_ALIGN;
    const size_t need = fa_weights_workspace_bytes();
    if (workspace_bytes < need) return FA_ERR_TOO_LARGE;
    const size_t nq = (size_t)B * Hq * T * D * 2, ns = (size_t)B * Hkv * cap * 4;
    const Range all[] = {range(out, ns), range(workspace, need), range(q, nq), range(lse, (size_t)B * Hq * T * 4),
                         range(cache->k, pool_bytes(cache)), range(cache->v, pool_bytes(cache)),
                         range(cache->table, (size_t)B * cache->max_pages * 4), range(cache->seq_len, (size_t)B * 4),
                         range(path, (size_t)B * T * 4), range(count, (size_t)B * 4),
                         range(weight, weight == out ? 0 : ns)};   // in place is fine, a partial overlap is not
    if (clash(all, sizeof(all) / sizeof(all[0]), 2)) return FA_ERR_ALIAS;
    st = fa::check_device();
    if (st != FA_OK) return st;

    const bool bf16 = cache->dtype == 0;
    WeighParams p;
    std::memset(&p, 0, sizeof(p));
    const int mode = path ? kPath : (T >= 128 ? kHeads : kRows);
    p.s = WeighShape{B, Hkv, group, T, mode, causal, NQ, mode == kHeads ? 256 : 128, cap, cache->seq_len, count};
    p.pages = pages_of(cache);
    p.q = q;
    p.lse = lse;
    p.path = path;
    p.weight = weight;
    p.out = out;
    p.cuts = static_cast<Cut *>(workspace);
    p.part = reinterpret_cast<float *>(p.cuts + kMaxCtas);
    p.box_rows = gcd(cache->page, 128);
    p.sl2 = (float)((double)scale * 1.4426950408889634);
    p.timeout_ns = timeout_ns;
    p.inject = inject;
    WeighMaps m;
    std::memset(&m, 0, sizeof(m));
    const long long eh[3] = {D, T, (long long)B * Hq}, er[3] = {D, rows, (long long)B * Hkv};
    if (!encode(&m.q, q, bf16, 3, mode == kHeads ? eh : er, NQ) || !encode_pool(&m.k, cache->k, q, cache, p.box_rows))
        return FA_ERR_TENSORMAP;
    return launch_weigh(D, bf16, m, p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

int fa_cache_weights(const fa_cache_t *cache, const void *q, const float *lse, const int32_t *path, const int32_t *count,
                     const float *weight, float *out, int Hq, int T, int causal, float scale, void *workspace,
                     size_t workspace_bytes, fa_stream_t stream)
{
    return fa_weights_debug(cache, q, lse, path, count, weight, out, Hq, T, causal, scale, workspace, workspace_bytes, stream, 0, 0);
}

size_t fa_evict_workspace_bytes(int B, int Hkv, int capacity, int keep)
{
    if (B < 1 || Hkv < 1 || keep < 1 || capacity <= keep) return 0;
    return (size_t)B * Hkv * (keep < capacity - keep ? keep : capacity - keep) * 2 * sizeof(uint2);
}

int fa_cache_evict(const fa_cache_t *cache, const float *weight, const int32_t *pos, float *weight_out, int32_t *pos_out,
                   int32_t *new_len, const int32_t *next_pos, int keep, int first, int last, void *workspace,
                   size_t workspace_bytes, fa_stream_t stream)
{
    int st = check_cache(cache);
    if (st != FA_OK) return st;
    const int B = cache->B, Hkv = cache->Hkv, cap = cache->max_pages * cache->page;
    if (keep < 1 || first < 0 || last < 0 || (long long)first + last > keep) return FA_ERR_BAD_DIM;
    if (B == 0) return FA_OK;
    if ((double)cache->num_pages * Hkv * cache->page > 4294967000.0) return FA_ERR_BAD_DIM;
    if ((long long)B * Hkv * 8 > 0x7fffffffLL || (double)keep * cache->D > 8.0 * 2147483647.0 - 65536.0) return FA_ERR_BAD_DIM;
    st = check_cache_pointers(cache);
    if (st != FA_OK) return st;
    const size_t need = fa_evict_workspace_bytes(B, Hkv, cap, keep);
    if (!new_len || (cap > 0 && (!weight || !pos || !weight_out || !pos_out)) || (last > 0 && !next_pos) || (need && !workspace))
        return FA_ERR_NULL_PTR;
    if (!aligned(weight, 4) || !aligned(pos, 4) || !aligned(weight_out, 4) || !aligned(pos_out, 4) || !aligned(new_len, 4) ||
        !aligned(next_pos, 4) || !aligned(workspace, 8))
        return FA_ERR_ALIGN;
    if (workspace_bytes < need) return FA_ERR_TOO_LARGE;
    const size_t ns = (size_t)B * Hkv * cap * 4;
    const Range all[] = {range(cache->k, pool_bytes(cache)), range(cache->v, pool_bytes(cache)), range(weight_out, ns), range(pos_out, ns),
                         range(new_len, (size_t)B * 4), range(workspace, need), range(weight, weight == weight_out ? 0 : ns),
                         range(pos, pos == pos_out ? 0 : ns), range(cache->table, (size_t)B * cache->max_pages * 4),
                         range(cache->seq_len, (size_t)B * 4), range(next_pos, (size_t)B * 4)};
    if (clash(all, sizeof(all) / sizeof(all[0]), 6)) return FA_ERR_ALIAS;
    st = fa::check_device();
    if (st != FA_OK) return st;
    EvictParams p;
    std::memset(&p, 0, sizeof(p));
    p.pages = pages_of(cache);
    p.k = static_cast<uint4 *>(cache->k);
    p.v = static_cast<uint4 *>(cache->v);
    p.seq_len = cache->seq_len;
    p.weight = weight;
    p.pos = pos;
    p.next_pos = next_pos;
    p.weight_out = weight_out;
    p.pos_out = pos_out;
    p.new_len = new_len;
    p.longest = keep < cap - keep ? keep : (cap > keep ? cap - keep : 0);
    p.from = static_cast<uint2 *>(workspace);
    p.to = p.from + (size_t)B * Hkv * p.longest;
    p.B = B;
    p.Hkv = Hkv;
    p.capacity = cap;
    p.chunks = cache->D / 8;
    p.keep = keep;
    p.first = first;
    p.last = last;
    return launch_evict(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

} // extern "C"
