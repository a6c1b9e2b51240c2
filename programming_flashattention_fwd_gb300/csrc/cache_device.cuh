// cache_device.cuh -- device code that the cache kernels share: finding a CTA's share of the work and
// the pages of a step's copies.
#pragma once
#include <cstdint>

#include "cache_internal.h"
#include "ptx.cuh"
#include "watchdog.cuh"

namespace fa {
namespace cache {

// Waits for the end of the kernels that this one may overlap (launch_overlapped): before the first access to
// memory that they may write, and before the first write that they may read or overwrite.  What they have written is
// read by ordinary loads: a non-coherent one is for data that nobody writes while the reading kernel runs, and
// this kernel runs since before those have ended.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// From here on the next kernel may be scheduled, once every CTA has come this far.
__device__ __forceinline__ void grid_done_soon() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct Share {
    int total, G;         // all steps, the CTAs that have some
    int b, off, left;     // this CTA's: `left` steps from step `off` of sequence b
};

// CTA `cta`'s share of the line of steps, steps(b) of them in sequence b: one warp adds up the
// lengths and finds the sequence that holds the share's first step.
template <typename Steps>
__device__ __forceinline__ Share find_share(int B, int lane, int cta, int grid, Steps steps)
{
    Share s;
    const int head = lane < B ? steps(lane) : 0;   // the first 32 sequences are looked up once
    int sum = head;
    for (int b = lane + 32; b < B; b += 32) sum += steps(b);
    sum = __reduce_add_sync(~0u, sum);
    s.total = sum;
    s.G = ctas(sum, grid, 1);
    const int at = cta + (lane & 1), edge = at < s.G ? cut(sum, s.G, at) : sum;   // both ends of the share at once
    const int begin = __shfl_sync(~0u, edge, 0);
    s.left = __shfl_sync(~0u, edge, 1) - begin;
    int before = 0;   // steps of the sequences before s.b
    for (s.b = 0; s.b < B; s.b += 32) {
        const int b = s.b + lane;
        const int mine = s.b == 0 ? head : (b < B ? steps(b) : 0);
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(~0u, upto, d);
            if (lane >= d) upto += x;
        }
        const uint32_t past = __ballot_sync(~0u, before + upto > begin);
        if (past) {
            const int src = __ffs(past) - 1;
            s.b += src;
            before += __shfl_sync(~0u, upto - mine, src);
            break;
        }
        before += __shfl_sync(~0u, upto, 31);
    }
    s.off = begin - before;
    return s;
}

// One probe of a phase by the whole (converged) warp, combined by a vote.
__device__ __forceinline__ bool mbar_try_all(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "vote.sync.all.pred q, p, 0xffffffff;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}

// A wait of the whole warp: usually the first probe succeeds (a few instructions instead of the
// bounded loop's), and every lane learns the same outcome.
struct WarpWait {
    volatile int *abort_flag;
    uint64_t timeout_ns;
    unsigned int *status;

    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, uint32_t site) const
    {
        if (mbar_try_all(bar, parity)) return true;
        return __all_sync(0xffffffffu, bounded_wait(bar, parity, abort_flag, timeout_ns, site, status)) != 0;
    }
};

// Place and phase of the next entry of a ring of N, without divisions.
template <int N>
struct Ring {
    uint32_t at = 0, phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++at == N) {
            at = 0;
            phase ^= 1;
        }
    }
};

// Page and row of slot `slot` of sequence b, as the table has it.  (Nothing is done with the number here, so
// that a look-up made ahead does not wait for it.)
__device__ __forceinline__ void page_of(const Pages &pg, int b, int slot, int &pid, int &row)
{
    const int at = slot / pg.page;
    row = slot - at * pg.page;
    pid = pg.table ? pg.table[(size_t)b * pg.max_pages + at] : b * pg.max_pages + at;
}

// A page that does not exist is given the number past the last, which a tensor map reads as zeros.
__device__ __forceinline__ int real_page(const Pages &pg, int pid) { return pid < 0 || pid >= pg.num_pages ? pg.num_pages : pid; }

// The pages of a sequence's boxes (box_rows slots each, a power of two of them to a key tile), 32 boxes at a time, a box
// to a lane, and the next 32 on their way: a look-up takes longer than a key tile.
struct PageRun {
    int page, row, next_page, next_row;

    __device__ __forceinline__ void look(const Pages &pg, int box_rows, int b, int n, int box, int &p, int &r)
    {
        const uint32_t slot = (uint32_t)box * box_rows;
        p = r = 0;
        if (slot < (uint32_t)n) page_of(pg, b, (int)slot, p, r);
        p = real_page(pg, p);
    }
    // box `first` is needed next, of boxes below `end`; `start`: the first one of a run
    __device__ __forceinline__ void at(const Pages &pg, int box_rows, int b, int n, int first, int end, int lane, bool start)
    {
        if (start) look(pg, box_rows, b, n, (first & ~31) + lane, page, row);
        if (!start && (first & 31) == 0) {
            page = next_page;
            row = next_row;
        }
        const int next = (first & ~31) + 32;
        if ((start || (first & 31) == 0) && next < end) look(pg, box_rows, b, n, next + lane, next_page, next_row);
    }
};

// The boxes 0 .. valid - 1 of a tile of keys, each of box_rows rows of one page and PANELS panels of 64 columns,
// global -> shared: lane `from` + i holds box i's page and row in it.  The whole warp calls it and one lane issues.
template <int PANELS>
__device__ __forceinline__ void load_boxes(uint32_t dst, uint32_t panel, uint32_t box, const CUtensorMap *m, int kvh, int page, int row, int from,
                                           int valid, uint32_t bar)
{
    const uint64_t map = reinterpret_cast<uint64_t>(m);
#pragma unroll (PANELS == 1 ? 2 : 1)   // short code for the start; D = 64 takes boxes twice as fast
    for (int i = 0; i < valid; ++i, dst += box) {
        const int p = __shfl_sync(~0u, page, from + i), r = __shfl_sync(~0u, row, from + i);
#pragma unroll
        for (int pn = 0; pn < PANELS; ++pn)
            asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                         "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                         " [%0], [%1, {%2, %3, %4, %5}], [%6];\n\t}" ::"r"(dst + pn * panel),
                         "l"(map), "r"(pn * 64), "r"(r), "r"(kvh), "r"(p), "r"(bar)
                         : "memory");
    }
}

} // namespace cache
} // namespace fa
