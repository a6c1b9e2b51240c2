// rotary_api.cpp -- fa_rotary and fa_rotary_append of include/fa.h: argument checks (before any CUDA call) and the launch.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "fa.h"
#include "fa_internal.h"
#include "rotary_internal.h"

namespace {

using fa::rotary::Params;

struct Range {
    uintptr_t at;
    size_t bytes;
};

Range range(const void *p, size_t bytes) { return Range{reinterpret_cast<uintptr_t>(p), p ? bytes : 0}; }
bool overlap(Range a, Range b) { return a.bytes && b.bytes && a.at < b.at + b.bytes && b.at < a.at + a.bytes; }
bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A [B, H, T, D] view, strides in elements; those of an extent of 1 do not count.
struct View {
    const void *data;
    long long n[3], s[3];
    long long D;
    size_t bytes() const
    {
        long long last = D;
        for (int i = 0; i < 3; ++i) last += (n[i] - 1) * s[i];
        return (size_t)last * 2;
    }
    bool empty() const { return n[0] == 0 || n[1] == 0 || n[2] == 0; }
};

View view(const fa_heads_t &h, int B, int T, int D)
{
    return View{h.data, {B, h.heads, T}, {B > 1 ? h.stride_b : 0, h.heads > 1 ? h.stride_h : 0, T > 1 ? h.stride_t : 0}, D};
}

// FA_OK, or what is wrong with the strides: negative or too large to address, or rows that are not on 16 bytes.
int check_view(const View &v)
{
    for (int i = 0; i < 3; ++i) {
        if (v.s[i] < 0 || (double)v.s[i] * (double)v.n[i] > 576460752303423488.0)   // 2^59: three of them are added up
            return FA_ERR_BAD_DIM;
        if (v.s[i] % 8 != 0) return FA_ERR_ALIGN;
    }
    return aligned(v.data, 16) ? FA_OK : FA_ERR_ALIGN;
}

// Whether no two elements of a view share their place: each stride steps over all that the smaller ones reach.
bool distinct(const View &v)
{
    int o[3] = {0, 1, 2};
    std::sort(o, o + 3, [&](int a, int b) { return v.s[a] < v.s[b]; });
    long long span = v.D;
    for (int i : o) {
        if (v.n[i] <= 1) continue;
        if (v.s[i] < span) return false;
        span += (v.n[i] - 1) * v.s[i];
    }
    return true;
}

bool same(const View &a, const View &b)
{
    return a.data == b.data && std::equal(a.n, a.n + 3, b.n) && std::equal(a.s, a.s + 3, b.s);
}

// Whether two views may share a place.  Apart in memory they do not; nor do heads of one tensor: the same strides from
// sequence to sequence and from token to token, and either, in a row, one view's heads after the other's, or all of them
// heads of a tensor whose heads are apart.
bool meet(const View &a, const View &b)
{
    if (!overlap(range(a.data, a.bytes()), range(b.data, b.bytes()))) return false;
    const View &x = a.data < b.data ? a : b, &y = a.data < b.data ? b : a;
    const long long gap = (long long)(reinterpret_cast<uintptr_t>(y.data) - reinterpret_cast<uintptr_t>(x.data)) / 2;
    if (x.s[0] != y.s[0] || x.s[2] != y.s[2]) return true;
    const long long wx = x.D + (x.n[1] - 1) * x.s[1], wy = y.D + (y.n[1] - 1) * y.s[1];
    if (wx <= gap && distinct(View{x.data, {x.n[0], 1, x.n[2]}, {x.s[0], 0, x.s[2]}, gap + wy})) return false;
    const long long sh = x.s[1] ? x.s[1] : y.s[1] ? y.s[1] : x.D;
    if ((x.s[1] && x.s[1] != sh) || (y.s[1] && y.s[1] != sh) || gap % sh != 0 || gap / sh < x.n[1]) return true;
    return !distinct(View{x.data, {x.n[0], gap / sh + y.n[1], x.n[2]}, {x.s[0], sh, x.s[2]}, x.D});
}

int check_table(const fa_rotary_table_t *r)
{
    if (!r) return FA_ERR_NULL_PTR;
    if (r->D != 64 && r->D != 128 && r->D != 256) return FA_ERR_UNSUPPORTED_D;
    if (r->rot < 0 || r->rot > r->D || r->rot % 2 != 0) return FA_ERR_BAD_DIM;
    if (r->interleaved != 0 && r->interleaved != 1) return FA_ERR_ARG;
    if (!std::isfinite(r->amplitude)) return FA_ERR_SCALE;
    return FA_OK;
}

// Fills the parameters that both entry points share; checks the views x[i] and y[i] of n segments, and against
// `others` (inputs, ranges that are not views).
int fill(Params &p, const fa_rotary_table_t *r, const fa_heads_t *x, const fa_heads_t *y, int n, int B, int T, const int32_t *start, const int32_t *position,
         const Range *others, int n_others)
{
    std::memset(&p, 0, sizeof(p));
    if (r->rot > 0 && !r->freq) return FA_ERR_NULL_PTR;
    if (!aligned(r->freq, 8) || !aligned(start, 4) || !aligned(position, 4)) return FA_ERR_ALIGN;
    View vx[3], vy[3];
    int heads = 0;
    for (int i = 0; i < n; ++i) {
        if (x[i].heads == 0) {
            vx[i] = vy[i] = View{nullptr, {0, 0, 0}, {0, 0, 0}, r->D};
        } else {
            if (!x[i].data) return FA_ERR_NULL_PTR;
            vx[i] = view(x[i], B, T, r->D);
            int st = check_view(vx[i]);
            if (st != FA_OK) return st;
            vy[i] = View{nullptr, {0, 0, 0}, {0, 0, 0}, r->D};
            if (y[i].data) {
                vy[i] = view(y[i], B, T, r->D);
                st = check_view(vy[i]);
                if (st != FA_OK) return st;
                if (!distinct(vy[i])) return FA_ERR_ALIAS;
            }
        }
        heads += x[i].heads;
        p.seg[i].x = vx[i].data;
        p.seg[i].y = const_cast<void *>(vy[i].data);
        p.seg[i].xb = vx[i].s[0];
        p.seg[i].xh = vx[i].s[1];
        p.seg[i].xt = vx[i].s[2];
        p.seg[i].yb = vy[i].s[0];
        p.seg[i].yh = vy[i].s[1];
        p.seg[i].yt = vy[i].s[2];
        p.seg[i].end = heads;
        p.seg[i].turned = i < 2;
    }
    for (int i = n; i < 3; ++i) p.seg[i].end = heads;
    const Range more[] = {range(r->freq, (size_t)(r->rot / 2) * 8), range(start, (size_t)B * 4), range(position, (size_t)B * T * 4)};
    for (int i = 0; i < n; ++i) {
        if (vy[i].empty()) continue;
        for (int j = 0; j < n; ++j) {
            // in place is fine: a thread reads its elements before it writes them
            if (!vx[j].empty() && !(i == j && same(vx[j], vy[i])) && meet(vy[i], vx[j])) return FA_ERR_ALIAS;
            if (i != j && !vy[j].empty() && meet(vy[i], vy[j])) return FA_ERR_ALIAS;
        }
        const Range w = range(vy[i].data, vy[i].bytes());
        for (const Range &o : more)
            if (overlap(w, o)) return FA_ERR_ALIAS;
        for (int j = 0; j < n_others; ++j)
            if (overlap(w, others[j])) return FA_ERR_ALIAS;
    }
    p.freq = r->freq;
    p.start = start;
    p.position = position;
    p.amplitude = r->amplitude;
    p.sign = 1.f;
    p.B = B;
    p.T = T;
    p.D = r->D;
    p.rot = r->rot;
    p.interleaved = r->interleaved;
    p.heads = heads;
    return FA_OK;
}

int check_heads(const fa_heads_t *x, const fa_heads_t *y, int n, int B, int T, int D)
{
    if (!x || !y) return FA_ERR_NULL_PTR;
    long long heads = 0;
    for (int i = 0; i < n; ++i) {
        if (x[i].heads < 0 || y[i].heads != x[i].heads) return FA_ERR_HEADS;
        heads += x[i].heads;
    }
    // blocks over heads, and over tokens, which are counted in 32 bits
    if (heads > 65535 || (double)B * T > 2147483647.0) return FA_ERR_BAD_DIM;
    return FA_OK;
}

} // namespace

extern "C" {

int fa_rotary(const fa_rotary_table_t *table, const fa_heads_t *x, const fa_heads_t *y, int n, int B, int T, const int32_t *start, const int32_t *position,
              int inverse, int dtype, fa_stream_t stream)
{
    int st = check_table(table);
    if (st != FA_OK) return st;
    if (n < 1 || n > 2 || (inverse != 0 && inverse != 1) || (dtype != 0 && dtype != 1) || (start && position)) return FA_ERR_ARG;
    if (B < 0 || T < 0) return FA_ERR_BAD_DIM;
    st = check_heads(x, y, n, B, T, table->D);
    if (st != FA_OK) return st;
    if (B == 0 || T == 0 || x[0].heads + (n > 1 ? x[1].heads : 0) == 0) return FA_OK;
    for (int i = 0; i < n; ++i)
        if (x[i].heads > 0 && !y[i].data) return FA_ERR_NULL_PTR;
    Params p;
    st = fill(p, table, x, y, n, B, T, start, position, nullptr, 0);
    if (st != FA_OK) return st;
    st = fa::check_device();
    if (st != FA_OK) return st;
    if (inverse) p.sign = -1.f;
    return fa::rotary::launch_rotary(p, dtype == 0, false, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

int fa_rotary_append(const fa_cache_t *cache, const fa_rotary_table_t *table, const fa_heads_t *x, const fa_heads_t *y, int T, const int32_t *start,
                     const int32_t *position, const int32_t *count, float *weight, int32_t *pos, fa_stream_t stream)
{
    int st = fa::cache::check_cache(cache);
    if (st != FA_OK) return st;
    st = check_table(table);
    if (st != FA_OK) return st;
    if (table->D != cache->D) return FA_ERR_UNSUPPORTED_D;
    if (start && position) return FA_ERR_ARG;
    if (T < 0) return FA_ERR_BAD_DIM;
    const int B = cache->B, Hkv = cache->Hkv;
    st = check_heads(x, y, 3, B, T, table->D);
    if (st != FA_OK) return st;
    if (x[1].heads != Hkv || x[2].heads != Hkv || x[0].heads % Hkv != 0) return FA_ERR_HEADS;
    if (B == 0 || T == 0) return FA_OK;
    st = fa::cache::check_cache_pointers(cache);
    if (st != FA_OK) return st;
    if (!aligned(count, 4) || !aligned(weight, 4) || !aligned(pos, 4)) return FA_ERR_ALIGN;
    const int cap = cache->max_pages * cache->page;
    const size_t ns = (size_t)B * Hkv * cap * 4, pool = (size_t)cache->num_pages * Hkv * cache->page * cache->D * 2;
    // the first four are written
    const Range all[] = {range(cache->k, pool), range(cache->v, pool), range(weight, ns), range(pos, ns), range(cache->table, (size_t)B * cache->max_pages * 4),
                         range(cache->seq_len, (size_t)B * 4), range(count, (size_t)B * 4), range(start, (size_t)B * 4), range(position, (size_t)B * T * 4),
                         range(table->freq, (size_t)(table->rot / 2) * 8)};
    const int n_all = sizeof(all) / sizeof(all[0]);
    Params p;
    st = fill(p, table, x, y, 3, B, T, start, position, all, n_all);
    if (st != FA_OK) return st;
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < n_all; ++j)
            if (i != j && overlap(all[i], all[j])) return FA_ERR_ALIAS;
        for (int j = 0; j < 3; ++j)
            if (x[j].heads > 0 && overlap(all[i], range(x[j].data, view(x[j], B, T, table->D).bytes()))) return FA_ERR_ALIAS;
    }
    st = fa::check_device();
    if (st != FA_OK) return st;
    p.seg[1].pool = 1;
    p.seg[2].pool = 2;
    p.pages = fa::cache::Pages{cache->table, cache->page, cache->max_pages, cache->num_pages};
    p.k = cache->k;
    p.v = cache->v;
    p.seq_len = cache->seq_len;
    p.count = count;
    p.weight = weight;
    p.pos = pos;
    p.Hkv = Hkv;
    p.capacity = cap;
    return fa::rotary::launch_rotary(p, cache->dtype == 0, true, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

} // extern "C"
