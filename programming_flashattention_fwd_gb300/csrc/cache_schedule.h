// cache_schedule.h -- how the cache kernels share out their work, used by the device code and by
// host-side checks of it.
//
// The work of a launch is a line of equal steps: sequence after sequence, in each its units one
// after another, in each unit its steps.  CTA c of G takes the steps [cut(c), cut(c + 1)) of the
// line, so that every CTA has the same number of steps whatever the sequences' lengths are; a unit
// that spans a cut is computed in parts and joined afterwards.  The lengths are read on the device,
// so a captured graph follows them.
#pragma once
#include <cstdint>

#include <cuda_runtime.h>

namespace fa {
namespace cache {

// ceil(a / b) for a >= 0, b > 0, a + b below 2^32 (32-bit arithmetic: the walks below run in every role)
__host__ __device__ __forceinline__ int cdiv(int a, int b) { return (int)(((uint32_t)a + (uint32_t)b - 1u) / (uint32_t)b); }
// a / b and ceil(a / b) for a >= 0 and a power of two b: a division costs a kernel's start some hundred cycles
__host__ __device__ __forceinline__ int shift_of(int b)
{
#ifdef __CUDA_ARCH__
    return 31 - __clz(b);
#else
    return __builtin_ctz((unsigned)b);
#endif
}
__host__ __device__ __forceinline__ int div2(int a, int b) { return a >> shift_of(b); }
__host__ __device__ __forceinline__ int cdiv2(int a, int b) { return (int)(((uint32_t)a + (uint32_t)b - 1u) >> shift_of(b)); }
__host__ __device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

// First step of CTA c when G CTAs share `total` steps (32-bit arithmetic while the product fits: the
// 64-bit division is some hundred cycles of a kernel's start).
__host__ __device__ __forceinline__ int cut(int total, int G, int c)
{
    if ((uint32_t)total < (1u << 23) && (uint32_t)c < 512u) return (int)((uint32_t)total * (uint32_t)c / (uint32_t)G);
    return (int)((long long)total * c / G);
}

// The CTA that has a step: the last one whose first step is not behind it.
__host__ __device__ __forceinline__ int cta_of(int total, int G, int step)
{
    if ((uint32_t)total < (1u << 23) && (uint32_t)G < 512u) return (int)(((uint32_t)(step + 1) * (uint32_t)G - 1u) / (uint32_t)total);
    return (int)(((long long)(step + 1) * G - 1) / total);
}

// CTAs that share `total` steps: at most `grid`, and no fewer than `least` steps each.
__host__ __device__ __forceinline__ int ctas(int total, int grid, int least)
{
    return clampi(total / least, 1, grid);
}

// ---------------------------------------------------------------- attention for drafted tokens
// A unit is one tile of `tile` rows (128, or 256: two row tiles side by side) of (sequence, KV head); its
// rows are (head in the group, token).  Its steps are the key tiles of the cache, then the key tiles of
// the drafted tokens.
struct TreeShape {
    int B, Hkv, T, rows;         // rows = (Hq / Hkv) * T
    int tile, units;             // units = tiles of `rows`
    int lbn;                     // log2 of the keys per step
    int capacity;                // slots of a sequence: max_pages * page
    const int32_t *seq_len;      // [B]
    const int32_t *draft_len;    // [B] or null: T
};

struct TreeLen {
    int n, t;        // cached slots, drafted tokens (clamped to what there is)
    int kc, nt;      // steps over the cache, all steps of a unit (0 without drafted tokens)
};

__host__ __device__ __forceinline__ TreeLen tree_len(const TreeShape &s, int b)
{
    TreeLen l;
    const int up = (1 << s.lbn) - 1;
    l.n = clampi(s.seq_len[b], 0, s.capacity);
    l.t = s.draft_len ? clampi(s.draft_len[b], 0, s.T) : s.T;
    l.kc = (l.n + up) >> s.lbn;
    l.nt = l.t > 0 ? l.kc + ((l.t + up) >> s.lbn) : 0;
    return l;
}

// One CTA's share of one unit: steps [k0, k1) of the unit's nt.
struct TreeSeg {
    int b, kvh, mt, k0, k1;
    TreeLen len;
};

// Walks a CTA's steps: `left` steps from step `off` of sequence b.
struct TreeWalk {
    int left, b, kvh, mt, k;
    TreeLen len;

    TreeWalk() = default;

    __host__ __device__ __forceinline__ TreeWalk(const TreeShape &s, int b0, int off, int steps) : left(steps), b(b0), kvh(0), mt(0), k(0)
    {
        if (left <= 0) return;
        len = tree_len(s, b);
        const int u = off / len.nt;
        k = off - u * len.nt;
        kvh = u / s.units;
        mt = u - kvh * s.units;
    }

    __host__ __device__ __forceinline__ bool next(const TreeShape &s, TreeSeg &g)
    {
        if (left <= 0) return false;
        if (mt == s.units) {
            mt = 0;
            if (++kvh == s.Hkv) {
                kvh = 0;
                do {
                    if (++b >= s.B) return false;
                    len = tree_len(s, b);
                } while (len.nt == 0);
            }
        }
        g.b = b;
        g.kvh = kvh;
        g.mt = mt;
        g.k0 = k;
        g.k1 = len.nt - k < left ? len.nt : k + left;
        g.len = len;
        left -= g.k1 - g.k0;
        k = 0;
        ++mt;
        return true;
    }
};

// Workspace slot of the part that CTA c computes of a unit it shares: a CTA shares at most the unit
// it starts in the middle of (slot 2 c) and the unit it leaves unfinished (slot 2 c + 1).
__host__ __device__ __forceinline__ int part_slot(int c, int k0) { return 2 * c + (k0 == 0 ? 1 : 0); }

// Parts of the unit (n steps) that CTA c's share starts in, at step k0 of it, if that is the unit's first cut
// (they are CTA c - 1's, c's and so on); else 0.
__host__ __device__ __forceinline__ int parts_from(int total, int G, int c, int k0, int n)
{
    if (k0 <= 0) return 0;
    const int u0 = cut(total, G, c) - k0;
    return cut(total, G, c - 1) > u0 ? 0 : cta_of(total, G, u0 + n - 1) - c + 2;
}

// ---------------------------------------------------------------- accumulated attention weight
// A unit is one key tile of `keys` slots of (sequence, KV head); its steps are the tiles of NQ query rows
// that see any of it.  The rows come in `planes` of a KV head:
//   heads    one plane a query head, rows in the order of their slots: with the causal mask the tiles
//            before the first row that sees the key tile are left out (long prompts)
//   rows     one plane with the rows of all heads of the group, head after head (short prompts)
//   path     one plane with the accepted rows only, gathered by index, head after head
enum WeighMode { kHeads = 0, kRows = 1, kPath = 2 };

struct WeighShape {
    int B, Hkv, group, T;
    int mode, causal;
    int NQ;                      // query rows of a step, a power of two
    int keys;                    // slots of a key tile: 256 in kHeads mode, else 128
    int capacity;
    const int32_t *seq_len;      // [B]
    const int32_t *count;        // [B] or null: T
};

struct WeighLen {
    int n, a;        // slots in use, query rows of a head
    int off;         // row i sees the slots below off + i + 1 (causal)
    int kt;          // units of a KV head: key tiles
    int rows, qt;    // rows of a plane, their tiles
    int planes;
    int per;         // tiles by which the first tile moves on from one key tile to the next (0: never)
    int w;           // key tile k starts at query tile max(0, per * k - w)
};

__host__ __device__ __forceinline__ WeighLen weigh_len(const WeighShape &s, int b)
{
    WeighLen l;
    l.n = clampi(s.seq_len[b], 0, s.capacity);
    l.a = s.count ? clampi(s.count[b], 0, s.T) : s.T;
    l.off = l.n - l.a;
    l.kt = cdiv2(l.n, s.keys);
    l.planes = s.mode == kHeads ? s.group : 1;
    l.rows = l.a == 0 ? 0 : (s.mode == kHeads ? l.a : (s.mode == kPath ? s.group * l.a : s.group * s.T));
    l.qt = cdiv2(l.rows, s.NQ);
    l.per = s.mode == kHeads && s.causal ? div2(s.keys, s.NQ) : 0;
    l.w = l.off >= 0 ? cdiv2(l.off, s.NQ) : -div2(-l.off, s.NQ);   // ceil(off / NQ)
    return l;
}

// First query tile of key tile k.
__host__ __device__ __forceinline__ int weigh_first(const WeighLen &l, int k)
{
    const int t = l.per * k - l.w;
    return l.per && t > 0 ? t : 0;
}

// Steps of key tile k; a key tile that no row sees has one, which adds nothing.
__host__ __device__ __forceinline__ int weigh_steps(const WeighLen &l, int k)
{
    return l.qt == 0 ? 1 : l.planes * (l.qt - weigh_first(l, k));
}

// Steps of the key tiles before k: with the first tile at max(0, per i - w), an arithmetic series.
__host__ __device__ __forceinline__ int weigh_before(const WeighLen &l, int k)
{
    if (l.qt == 0) return k;
    long long skipped = 0;
    if (l.per) {
        const int i0 = l.w <= 0 ? 0 : cdiv2(l.w, l.per);   // first key tile with per i >= w
        if (k > i0) {
            const long long m = k - i0;
            skipped = (long long)l.per * (i0 + (k - 1)) * m / 2 - (long long)l.w * m;
        }
    }
    return (int)(l.planes * ((long long)k * l.qt - skipped));
}

// One CTA's share of one unit: steps [s0, s1) of the ns of key tile kt.
struct WeighSeg {
    int b, kvh, kt, s0, s1, ns, first;
    WeighLen len;
};

// The plane and the query tile of a segment's steps, one after another.
struct WeighTiles {
    int plane, qt, first, end;

    __host__ __device__ __forceinline__ explicit WeighTiles(const WeighSeg &g) : first(g.first), end(g.len.qt)
    {
        const int per = end - first;
        plane = per > 0 && g.s0 ? g.s0 / per : 0;
        qt = per > 0 ? first + g.s0 - plane * per : 0;
    }
    __host__ __device__ __forceinline__ void next()
    {
        if (++qt >= end) {
            qt = first;
            ++plane;
        }
    }
};

// One CTA's share of one head where all key tiles have the same steps (kRows, kPath): `steps` of them, from
// step s of key tile kt, ns to a key tile.
struct WeighRun {
    int b, kvh, kt, s, steps, ns;
    WeighLen len;
};

// Walks a CTA's steps: `left` of them from step `s` of key tile kt.  The lengths are looked up and
// the first key tile is searched for once a sequence, not once a key tile: a drafting step has one
// step a key tile.
struct WeighWalk {
    int left, b, kvh, kt, s;
    WeighLen len;

    WeighWalk() = default;

    // `steps` steps from step `off` of sequence b0
    __host__ __device__ __forceinline__ WeighWalk(const WeighShape &sh, int b0, int off, int steps) : left(steps), b(b0), kvh(0), kt(0), s(0)
    {
        if (left <= 0) return;
        len = weigh_len(sh, b);
        const int one = weigh_before(len, len.kt);
        kvh = off / one;
        const int in = off - kvh * one;
        int hi = len.kt - 1;
        if (!len.per) kt = hi = in / weigh_steps(len, 0);
        while (kt < hi) {   // the key tile that holds step `in` of the head
            const int mid = (kt + hi + 1) / 2;
            if (weigh_before(len, mid) <= in)
                kt = mid;
            else
                hi = mid - 1;
        }
        s = in - weigh_before(len, kt);
    }

    // to the next head that has key tiles, behind the last one of a head
    __host__ __device__ __forceinline__ bool settle(const WeighShape &sh)
    {
        if (left <= 0) return false;
        if (kt == len.kt) {
            kt = 0;
            if (++kvh == sh.Hkv) {
                kvh = 0;
                do {
                    if (++b >= sh.B) return false;
                    len = weigh_len(sh, b);
                } while (len.kt == 0);
            }
        }
        return true;
    }

    // a head at a time (kRows, kPath): a drafting step has one step a key tile, and what is done for each
    // key tile is what bounds it
    __host__ __device__ __forceinline__ bool next_run(const WeighShape &sh, WeighRun &r)
    {
        if (!settle(sh)) return false;
        r.b = b;
        r.kvh = kvh;
        r.kt = kt;
        r.s = s;
        r.len = len;
        r.ns = len.qt > 0 ? len.qt : 1;
        const int all = (len.kt - kt) * r.ns - s;
        r.steps = all < left ? all : left;
        left -= r.steps;
        kt = len.kt;
        s = 0;
        return true;
    }

    __host__ __device__ __forceinline__ bool next(const WeighShape &sh, WeighSeg &g)
    {
        if (!settle(sh)) return false;
        g.b = b;
        g.kvh = kvh;
        g.kt = kt;
        g.len = len;
        g.first = weigh_first(len, kt);
        g.ns = len.qt == 0 ? 1 : len.planes * (len.qt - g.first);
        g.s0 = s;
        g.s1 = g.ns - s < left ? g.ns : s + left;
        left -= g.s1 - g.s0;
        s = 0;
        ++kt;
        return true;
    }
};

} // namespace cache
} // namespace fa
