// bwd_internal.h -- the work of attention's backward pass: its parameters and the schedule of its kernels, shared
// by the host API (bwd_api.cpp), the kernels (bwd_sm103.cu) and host-side checks.  Not part of the public ABI.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "schedule.h"

namespace fa {
namespace bwd {

// What a kernel accumulates while it streams tiles past a resident tile of 128 rows:
//   kQ   dQ of 128 queries, past the keys they see
//   kKV  dK and dV of 128 keys, past the queries (of every query head of the group) that see them
//   kK, kV  dK or dV alone: at D = 256 both accumulators together would fill tensor memory
enum Mode { kQ = 0, kKV = 1, kK = 2, kV = 3 };

constexpr int kRows = 128;                                         // resident rows
constexpr int step_rows(int D) { return D == 256 ? 64 : 128; }     // streamed rows of a step
constexpr int kMaxParts = 160;   // parts of cut units that a workspace has room for

// One kernel's line of work: units of (head plane, tile of 128 resident rows), each cut into `parts` runs of
// its steps.  A step is one tile of step_rows streamed rows.
struct Shape {
    int rows, cols;       // resident and streamed rows of a head: (Sq, Sk) or (Sk, Sq)
    int heads, group;     // resident heads of a sequence; query heads of a KV head
    int coff;             // key j is seen by query i iff j <= i + coff
    int causal;
    int tiles, steps;     // tiles of resident rows, of streamed rows
    int planes;           // B * heads
    int parts, num;       // parts of a unit; planes * tiles * parts
    FastDiv f_planes, f_tiles, f_heads, f_group, f_parts;
};

struct Unit {
    int z, t;             // resident plane and tile
    int n;                // steps of this part
    int plane, tile;      // streamed plane and tile of its first step
    int first, end;       // streamed tiles of a plane: [first, end)
    int slot;             // (unit, part): where a cut unit's part is left
};

// Steps of the tile t: [first, end) of each streamed plane.
template <bool ROWQ, int BN>
__host__ __device__ __forceinline__ void seen(const Shape &s, int t, int &first, int &end)
{
    first = 0;
    end = s.steps;
    if (!s.causal) return;
    if (ROWQ) {          // keys up to the last one that the tile's last row sees
        const long long hi = (long long)t * kRows + (kRows - 1) + s.coff;
        const long long n = hi < 0 ? 0 : hi / BN + 1;
        if (n < end) end = (int)n;
    } else {             // queries from the first one that sees the tile's first key
        const long long lo = (long long)t * kRows - s.coff;
        const long long i = lo < 0 ? 0 : lo / BN;
        first = i < end ? (int)i : end;
    }
}

// The unit that CTA c of G takes in `round`; false where it has no more.  With a mask the heaviest tiles come first
// (the last queries, the first keys), without one neighbouring units share the streamed heads.
template <bool ROWQ, int BN>
__host__ __device__ __forceinline__ bool unit_at(const Shape &s, int G, int c, int round, Unit &u)
{
    const long long g64 = unit_index(G, c, round);
    if (g64 >= s.num) return false;
    const uint32_t g = (uint32_t)g64, w = fdiv(g, s.f_parts);
    const int part = (int)(g - w * s.f_parts.d);
    if (s.causal) {
        const uint32_t q = fdiv(w, s.f_planes);
        u.t = ROWQ ? s.tiles - 1 - (int)q : (int)q;
        u.z = (int)(w - q * s.f_planes.d);
    } else {
        const uint32_t q = fdiv(w, s.f_tiles);
        u.z = (int)q;
        u.t = (int)(w - q * s.f_tiles.d);
    }
    const int b = (int)fdiv((uint32_t)u.z, s.f_heads), h = u.z - b * s.heads;
    seen<ROWQ, BN>(s, u.t, u.first, u.end);
    const int per = u.end - u.first;
    const long long all = ROWQ ? per : (long long)per * s.group;
    const int n0 = (int)(all * part / s.parts), n1 = (int)(all * (part + 1) / s.parts);
    u.n = n1 - n0;
    const int skip = per > 0 ? n0 / per : 0;
    u.plane = ROWQ ? b * (s.heads / s.group) + (int)fdiv((uint32_t)h, s.f_group) : u.z * s.group + skip;
    u.tile = u.first + (ROWQ ? n0 : n0 - skip * per);
    u.slot = (u.z * s.tiles + u.t) * s.parts + part;
    return true;
}

inline void set_divisors(Shape &s)
{
    s.f_planes = make_fastdiv((uint32_t)s.planes);
    s.f_tiles = make_fastdiv((uint32_t)s.tiles);
    s.f_heads = make_fastdiv((uint32_t)s.heads);
    s.f_group = make_fastdiv((uint32_t)s.group);
    s.f_parts = make_fastdiv((uint32_t)s.parts);
}

// The shape of a kernel's work.  Where the units alone would leave SMs idle, their steps are cut into parts, as
// many as fit kMaxParts slots and leave at least two steps to a part.
inline Shape make_shape(bool rowq, int B, int Hq, int Hkv, int Sq, int Sk, int D, int causal)
{
    Shape s = {};
    const int BN = step_rows(D);
    s.rows = rowq ? Sq : Sk;
    s.cols = rowq ? Sk : Sq;
    s.heads = rowq ? Hq : Hkv;
    s.group = Hq / Hkv;
    s.coff = causal == 2 ? Sk - Sq : 0;
    s.causal = causal != 0;
    s.tiles = (s.rows + kRows - 1) / kRows;
    s.steps = (s.cols + BN - 1) / BN;
    s.planes = B * s.heads;
    const long long units = (long long)s.planes * s.tiles, longest = (long long)s.steps * (rowq ? 1 : s.group);
    s.parts = 1;
    if (units > 0 && units * 2 <= kMaxParts) {
        const long long most = kMaxParts / units, able = longest / 2;
        s.parts = (int)(most < able ? most : able);
        if (s.parts < 1) s.parts = 1;
    }
    s.num = (int)(units * s.parts);
    set_divisors(s);
    return s;
}

struct Params {
    Shape s;
    const float *nl, *dc;    // [B * Hq][pad] -lse log2 e + shift, and delta 2^-shift; rows at or behind Sq: -inf, 0
    int pad;                 // Sq rounded up to 128
    void *out, *out_v;       // dq, or dk and dv
    float *part, *part_v;    // [slots][128][D] sums of cut units (parts > 1)
    float sl2;               // scale log2 e
    float dscale;            // 2^-shift
    float out_scale, out_v_scale;
    uint32_t al32;           // outputs are 32-byte aligned
    uint32_t first;          // the first kernel behind lse and delta
    uint64_t timeout_ns;
    uint32_t inject;         // fault injection: the first second tile is never loaded (bit 0: in every CTA, bit 1: in CTA 0)
};

// The operands: resident first and second (q and do, or k and v), streamed first and second (k and v, or q and do).
struct Maps {
    CUtensorMap r1, r2, s1, s2;
};

cudaError_t launch_prep(const void *o, const void *d_o, const float *lse, const float *dlse, float *nl, float *dc, long long planes, int Sq, int pad, int D,
                        bool bf16, float shift, cudaStream_t st);
cudaError_t launch_bwd(int mode, int D, bool bf16, const Maps &m, const Params &p, cudaStream_t st);
// out [planes, rows, D] = round(scale * sum of the parts)
cudaError_t launch_join(const float *part, void *out, const Shape &s, int D, bool bf16, float scale, cudaStream_t st);
cudaError_t read_and_clear_bwd_status(uint32_t *word);

} // namespace bwd
} // namespace fa
