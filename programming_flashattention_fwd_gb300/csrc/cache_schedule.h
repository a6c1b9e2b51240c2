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

__host__ __device__ __forceinline__ int cdiv(int a, int b) { return (int)(((long long)a + b - 1) / b); }
__host__ __device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

// First step of CTA c when G CTAs share `total` steps.
__host__ __device__ __forceinline__ int cut(int total, int G, int c) { return (int)((long long)total * c / G); }

// CTAs that share `total` steps: at most `grid`, and no fewer than `least` steps each.
__host__ __device__ __forceinline__ int ctas(int total, int grid, int least)
{
    return clampi(total / least, 1, grid);
}

// ---------------------------------------------------------------- attention for drafted tokens
// A unit is one 128-row tile of (sequence, KV head); its rows are (head in the group, token).
// Its steps are the key tiles of the cache, then the key tiles of the drafted tokens.
struct TreeShape {
    int B, Hkv, T, rows;         // rows = (Hq / Hkv) * T
    int mtiles;                  // 128-row tiles of `rows`
    int BN;                      // keys per step
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
    l.n = clampi(s.seq_len[b], 0, s.capacity);
    l.t = s.draft_len ? clampi(s.draft_len[b], 0, s.T) : s.T;
    l.kc = cdiv(l.n, s.BN);
    l.nt = l.t > 0 ? l.kc + cdiv(l.t, s.BN) : 0;
    return l;
}

// One CTA's share of one unit: steps [k0, k1) of the unit's nt.
struct TreeSeg {
    int b, kvh, mt, k0, k1;
    TreeLen len;
};

// Walks a CTA's steps: `left` steps from step `off` of sequence b.
struct TreeWalk {
    int b, off, left;

    __host__ __device__ __forceinline__ bool next(const TreeShape &s, TreeSeg &g)
    {
        while (left > 0 && b < s.B) {
            const TreeLen l = tree_len(s, b);
            const int per = s.Hkv * s.mtiles * l.nt;
            if (off >= per) {
                off -= per;
                ++b;
                continue;
            }
            const int u = off / l.nt;
            g.b = b;
            g.kvh = u / s.mtiles;
            g.mt = u - g.kvh * s.mtiles;
            g.k0 = off - u * l.nt;
            g.k1 = l.nt - g.k0 < left ? l.nt : g.k0 + left;
            g.len = l;
            off += g.k1 - g.k0;
            left -= g.k1 - g.k0;
            return true;
        }
        return false;
    }
};

// Workspace slot of the part that CTA c computes of a unit it shares: a CTA shares at most the unit
// it starts in the middle of (slot 2 c) and the unit it leaves unfinished (slot 2 c + 1).
__host__ __device__ __forceinline__ int part_slot(int c, int k0) { return 2 * c + (k0 == 0 ? 1 : 0); }

} // namespace cache
} // namespace fa
