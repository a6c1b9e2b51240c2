// tree_sm103.cu -- attention of drafted tokens over a paged key/value cache (fa_tree_fwd).
//
// For sequence b, KV head c, drafted token t and each query head h of c's group:
//
//     s_j = scale q.k_j over the n_b cached slots and the drafted tokens j on t's path to its root
//     o   = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),   lse = m + ln sum_j exp(s_j - m)
//
// The rows of one KV head (heads of the group x drafted tokens, consecutive in memory) are packed
// into 128-row tiles, so that K and V are read once for all of them.  A key costs 4 D flops a row and
// 4 D bytes: with fewer than about 280 rows the read bounds the kernel.  The keys of every unit
// (sequence, KV head, row tile) are cut so that each CTA has the same number of key steps
// (cache_schedule.h); a unit that is cut leaves normalised fp32 partial rows with their log-sum-exp in
// the workspace and a second kernel joins them in the order of the keys, the same on every run.
// (Joined by the last CTA to arrive instead, with counters and fences: one token over 4096 slots 24.8
// instead of 17 us, 8 x 64 tokens over 16384 138 instead of 102, when these calls took that long; they take 10.7 and 93
// now, and the comparison has not been made again.)
//
// Measured, 8 sequences, 32 heads over 8 KV heads, bf16, of 6.8 TB/s copied:
//     D = 64, 131072 slots    one token 6.8 TB/s, 32 tokens 6.7     D = 256, 65536 slots   7.2, 7.1
//     D = 128, 131072 slots   one token 7.0 TB/s (16-slot pages too), 32 tokens 6.9, 64 tokens (256 rows,
//                             where the softmax is as busy as memory) 6.1
// Short calls are a chain of latencies (start, one unit, second kernel): one sequence, one token, 10 us
// over 16 slots and 11 over 4096.  So are many short units, about 3 us each of an SM's time, which
// the reads of the next one only partly cover: 64 x 128 slots 23 us, 64 x 512 39 (3.4 TB/s), 64 x 1024 52 (5.1), 64 x
// 4096 171 (6.3).
//
// Per CTA (one per SM):
//   warps 0, 3    K and V producers (one warp for both: 5.5 instead of 6.4 TB/s at D = 64, 4.9 instead of
//                 6.4 with 16-slot pages): per step one TMA box per page and 64-column panel, into one ring of NS
//                 slots in the order in which the products take them (K_0, K_1, V_0, K_2, V_1, ...).  Pages are looked
//                 up 32 boxes ahead (a step ahead: with 16-slot pages 189 instead of 179 us over 8 x 65536 slots at
//                 D = 64, 323 instead of 314 at 128).  Warp 3 finds the CTA's share first.
//   warp 1        TMEM owner and MMA issuer: S = Q K^T, O += P V (tcgen05, fp32 in tensor memory)
//   warp 2        Q producer
//   warps 4-7,    softmax, one thread per row, in two groups (one at D = 256) so that one group's softmax
//   warps 8-11    runs beside the other's matrix products:
//     up to 128 rows    the groups take alternate key steps, each with its own running maximum, sum and O;
//                       they are joined in the epilogue, where both read both accumulators (half of
//                       the columns each)
//     more (PAIR)       each group has a row tile of its own and takes every step: K and V are read once
//                       for 256 rows (8 x 64 tokens over up to 16384 slots 102 us, now 93; a row tile by itself 139)
//     D = 256           one group, 64-key steps (two accumulators do not fit); the other reads half of the result
//
// Tensor memory: S_0, S_1 (BN columns each; P, 16-bit, overwrites its S), then the accumulators.
//
// Keys that a row must not see: scores are replaced by -inf, not summed with it, and the V rows
// behind the last valid key of a step are zeroed in shared memory before P V, so that neither
// what the cache holds behind a sequence's end nor its page's old contents reach the result.
// Non-finite values in a drafted token's V are taken out of the matrix product and added, as what
// they are, to the rows that see that token, so that they do not leak into other branches.
#include <atomic>
#include <cstdint>

#include "cache_device.cuh"
#include "cache_internal.h"
#include "ptx.cuh"
#include "watchdog.cuh"

namespace fa {

__device__ unsigned int g_tree_status;

namespace cache {

namespace {

constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;
constexpr float kTau = 12.f;   // O is rescaled when the maximum grows by more than this (log2 units): P <= 4096 fits fp16

enum Site : uint32_t {
    S_EMPTY = 1, S_Q = 2, S_FULL = 3, S_P = 4, S_S = 5, S_PV = 6, S_DRAIN = 7, S_QFREE = 8, S_SMEM = 9, S_JOIN = 10, S_READ = 11
};

template <int D, bool PAIR>
struct Cfg {
    static constexpr int LBN = D == 256 ? 6 : 7, BN = 1 << LBN;
    static constexpr int NG = D == 256 ? 1 : 2;          // groups that take key steps, of the two that read the result
    static constexpr int STRIDE = PAIR ? 1 : NG;         // key steps from one of a group to its next
    static constexpr int THREADS = 128 + 128 * 2;
    static constexpr int PANELS = D / 64;
    static constexpr int QTILE = PANELS * 16384;         // one tile of 128 rows, or two of up to 64
    static constexpr int QAREA = PAIR ? 2 * QTILE : QTILE;
    static constexpr int KVPANEL = BN * 128, KVTILE = PANELS * KVPANEL;
    // 160 or 192 KB of K / V in flight (6 slots, against 5: 6.76 and 6.7 TB/s over a long cache at D = 128)
    static constexpr int NS = D == 64 ? 12 : (D == 128 && !PAIR ? 6 : 5);
    static constexpr int OFF_RING = QAREA;
    static constexpr int OFF_BAR = OFF_RING + NS * KVTILE;
    static constexpr int NBAR = 4 + 2 * NS + 2 + 2 + 2 + 2 + 1;    // q[2], qfree[2], full, empty, S[2], P[2], PV[2], join, read, done
    static constexpr int OFF_ML = OFF_BAR + ((NBAR * 8 + 15) / 16) * 16;   // [2][128] (m, l)
    static constexpr int OFF_MISC = OFF_ML + 2 * 128 * 8;
    static constexpr int BYTES = OFF_MISC + 64;
    static_assert(BYTES <= 232448, "shared memory of one CTA");
    // room to align the base to 1024 bytes, as far as there is any (the kernel checks what it got)
    static constexpr int ALLOC = BYTES + 1024 <= 232448 ? BYTES + 1024 : 232448;
    static constexpr uint32_t COL_O = 2 * BN;
    static_assert(2 * BN + NG * D <= 512, "tensor-memory columns");
    static_assert(!PAIR || NG == 2, "two row tiles, two groups");
};

struct Misc {
    uint32_t tmem;
    int abort;
    int nonfinite;      // 1 + index of the last segment whose drafted V held a non-finite value
    TreeWalk share;     // this CTA's share, not walked yet
};

// x is an infinity or a NaN, in a 16-bit pair: the pair with those halves cleared, and whether there were any.
template <bool BF16>
__device__ __forceinline__ uint32_t drop_nonfinite(uint32_t w, bool &any)
{
    constexpr uint32_t E = BF16 ? 0x7f80u : 0x7c00u;
    const bool lo = (w & E) == E, hi = ((w >> 16) & E) == E;
    any |= lo | hi;
    return (lo ? 0u : (w & 0xffffu)) | (hi ? 0u : (w & 0xffff0000u));
}

template <bool BF16>
__device__ __forceinline__ float half_to_float(uint16_t h)
{
    if constexpr (BF16) {
        return __uint_as_float((uint32_t)h << 16);
    } else {
        float f;
        asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(h));
        return f;
    }
}

// Bits of the drafted tokens lo .. lo + 32 W - 1 that token t sees: its path to the root (parents
// come before their children; an entry that does not ends the path).
template <int W>
__device__ __forceinline__ void path_bits(const int32_t *parent, int t, int lo, uint32_t (&bits)[W])
{
#pragma unroll
    for (int w = 0; w < W; ++w) bits[w] = 0;
    if (!parent) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int c = t - lo - 32 * w;   // keys up to lo + 32 w + c
            bits[w] = c < 0 ? 0u : (c >= 31 ? ~0u : (2u << c) - 1u);
        }
        return;
    }
    for (int j = t; j >= lo;) {
        const int i = j - lo;
#pragma unroll
        for (int w = 0; w < W; ++w)
            if ((i >> 5) == w) bits[w] |= 1u << (i & 31);
        const int up = parent[j];
        if (up >= j) break;
        j = up;
    }
}

// Steps of sequence b.
__device__ __forceinline__ int tree_steps(const TreeShape &s, int b) { return s.Hkv * s.units * tree_len(s, b).nt; }

// NaN into every row of a CTA's share, its parts included: threads `first`, first + step, ... take a row each.
template <int D>
__device__ __forceinline__ void leave_nan(const TreeParams &p, TreeWalk walk, int first, int step)
{
    const float nan = __uint_as_float(~0u);
    TreeSeg g;
    while (walk.next(p.s, g)) {
        for (int urow = first; urow < p.s.tile; urow += step) {
            const int row = g.mt * p.s.tile + urow;
            if (row >= p.s.rows || row % p.s.T >= g.len.t) continue;
            if (g.k0 == 0 && g.k1 == g.len.nt) {
                const size_t orow = (size_t)(g.b * p.s.Hkv + g.kvh) * p.s.rows + row;
                for (int c = 0; c < D * 2; c += 16)
                    st_global_v4(static_cast<uint8_t *>(p.o) + orow * D * 2 + c, ~0u, ~0u, ~0u, ~0u);
                p.lse[orow] = nan;
            } else {
                const size_t prow = (size_t)part_slot(blockIdx.x, g.k0) * p.part_rows + urow;
                for (int c = 0; c < D; ++c) p.part_o[prow * D + c] = nan;
                p.part_lse[prow] = nan;
            }
        }
    }
}

// For the joining kernel: the cut unit that the share starts in, if the unit's first cut is there.
__device__ __forceinline__ Cut cut_of(const TreeWalk &walk, int total, int ctas)
{
    Cut c = {};
    if (walk.left > 0) c = Cut{walk.b, walk.kvh, walk.mt, parts_from(total, ctas, blockIdx.x, walk.k, walk.len.nt), walk.len.t, {}};
    return c;
}

// A CTA that the alignment of its shared memory leaves no room in: it does nothing but what the joining kernel and the
// caller rely on, without shared memory (each warp looks the share up for itself).
template <int D>
__device__ __noinline__ void no_room(const TreeParams &p)
{
    grid_wait();
    const Share w = find_share(p.s.B, threadIdx.x & 31, blockIdx.x, gridDim.x, [&](int b) { return tree_steps(p.s, b); });
    const TreeWalk mine(p.s, w.b, w.off, w.left);
    if (threadIdx.x == 0) {
        atomicOr(&g_tree_status, 1u | (S_SMEM << 8));
        p.cuts[blockIdx.x] = cut_of(mine, w.total, w.G);
    }
    leave_nan<D>(p, mine, threadIdx.x, blockDim.x);
}

template <int D, bool BF16, bool PAIR>
__global__ void __launch_bounds__(Cfg<D, PAIR>::THREADS, 1)
    tree_kernel(const __grid_constant__ TreeMaps maps, const __grid_constant__ TreeParams p)
{
    using C = Cfg<D, PAIR>;
    constexpr int BN = C::BN, NG = C::NG;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sb = raw + pad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sRing = sb + C::OFF_RING, bar0 = sb + C::OFF_BAR;
    auto bar_q = [&](uint32_t i) { return bar0 + 8u * i; };
    auto bar_qfree = [&](uint32_t i) { return bar0 + 16u + 8u * i; };
    auto bar_full = [&](uint32_t s) { return bar0 + 8u * (4 + s); };
    auto bar_empty = [&](uint32_t s) { return bar0 + 8u * (4 + C::NS + s); };
    const uint32_t barS = bar0 + 8u * (4 + 2 * C::NS), barP = barS + 16, barPV = barS + 32, barJoin = barS + 48,
                   barRead = barS + 56, barDone = barS + 64;
    float2 *ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
    volatile Misc *misc = reinterpret_cast<volatile Misc *>(smem + C::OFF_MISC);
    volatile int *abort_flag = &misc->abort;
    unsigned int *status = &g_tree_status;
    const uint64_t tmo = p.timeout_ns;

    grid_done_soon();
    if (pad + (uint32_t)C::BYTES > dynamic_smem_size_u32() || (p.inject & 4u)) {
        no_room<D>(p);
        return;
    }
    int total = 0, ctas = 1;   // (warp 3) all steps, the CTAs that share them
    if (warp == 0) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(bar_q(i), 1);
                mbar_init(bar_qfree(i), 1);
                mbar_init(barS + 8 * i, 1);
                mbar_init(barP + 8 * i, 4);
                mbar_init(barPV + 8 * i, 1);
            }
            for (int s = 0; s < C::NS; ++s) {
                mbar_init(bar_full(s), 1);
                mbar_init(bar_empty(s), 1);
            }
            mbar_init(barJoin, 8);
            mbar_init(barRead, 8);
            mbar_init(barDone, 1);
            misc->abort = 0;
            misc->nonfinite = 0;
            fence_mbar_init();
        }
    } else if (warp == 1) {
        tmem_alloc(smem_u32(const_cast<uint32_t *>(&misc->tmem)), 512);
        tmem_relinquish();
    } else if (warp == 2) {
        if (lane < 5) tma_prefetch_map(lane == 0 ? &maps.q : lane == 1 ? &maps.k : lane == 2 ? &maps.v : lane == 3 ? &maps.k_new : &maps.v_new);
    } else if (warp == 3) {
        grid_wait();
        const Share w = find_share(p.s.B, lane, blockIdx.x, gridDim.x, [&](int b) { return tree_steps(p.s, b); });
        const TreeWalk mine(p.s, w.b, w.off, w.left);
        total = w.total;
        ctas = w.G;
        if (lane == 0) const_cast<Misc *>(misc)->share = mine;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_wait();   // every thread: what it reads and writes from here on may be the kernel's before
    const uint32_t tmem = misc->tmem;
    TreeWalk walk = const_cast<const Misc *>(misc)->share;
    TreeSeg g = {};
    const WarpWait wait_all{abort_flag, tmo, status};

    // keys of step kt that there are
    auto valid_of = [&](const TreeSeg &g, int kt) {
        return kt < g.len.kc ? min(BN, g.len.n - kt * BN) : min(BN, g.len.t - (kt - g.len.kc) * BN);
    };

    if (warp == 0 || warp == 3) {
        // ------------------------------------------------------------ K producer, V producer
        const bool is_v = warp == 3;
        const CUtensorMap *pool = is_v ? &maps.v : &maps.k, *fresh = is_v ? &maps.v_new : &maps.k_new;
        const int boxes = div2(BN, p.box_rows);       // boxes of a step (one panel)
        int use0 = 0, last = 0;                       // the segment's first place in the ring, this warp's last
        uint32_t issued = 0;                          // bit i: place last - i is this warp's
        if (is_v && lane == 0) p.cuts[blockIdx.x] = cut_of(walk, total, ctas);
        bool skip = is_v && ((p.inject & 1u) || ((p.inject & 2u) && blockIdx.x == 0));
        bool ok = true;
        PageRun run;
        while (ok && walk.next(p.s, g)) {
            const int nk = g.k1 - g.k0;
            for (int j = 0; j < nk; ++j) {
                const int kt = g.k0 + j;
                run.at(p.pages, p.box_rows, g.b, g.len.n, kt * boxes, g.k1 * boxes, lane, j == 0);
                // K_0, K_1, V_0, K_2, V_1, ..., V_last
                const int use = use0 + (is_v ? (j + 1 < nk ? 2 * j + 2 : 2 * j + 1) : (j ? 2 * j - 1 : 0));
                const uint32_t at = (uint32_t)use % C::NS, bar = bar_full(at), dst = sRing + at * C::KVTILE;
                ok = wait_all(bar_empty(at), (((uint32_t)use / C::NS) & 1) ^ 1, S_EMPTY);
                if (!ok) break;
                if (skip) {
                    skip = false;
                    continue;
                }
                if (kt < g.len.kc) {
                    const int valid = min(boxes, cdiv2(g.len.n - kt * BN, p.box_rows));
                    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(valid * p.box_rows * 128 * C::PANELS));
                    __syncwarp();
                    load_boxes<C::PANELS>(dst, C::KVPANEL, p.box_rows * 128, pool, g.kvh, run.page, run.row, kt * boxes & 31, valid, bar);
                } else {
                    if (lane == 0) mbar_arrive_expect_tx(bar, C::KVTILE);
                    __syncwarp();
                    if (lane < C::PANELS)
                        tma_load_3d(dst + lane * C::KVPANEL, fresh, lane * 64, (kt - g.len.kc) * BN, g.b * p.s.Hkv + g.kvh, bar);
                }
                issued = (issued << (use - last)) | 1u;
                last = use;
            }
            use0 += 2 * nk;
        }
        // after an abort nobody else waits for the loads in flight: they land before the CTA ends
        if (lane == 0 && *abort_flag)
            for (int i = 0; i < C::NS; ++i)
                if ((issued >> i) & 1u)
                    bounded_wait(bar_full((uint32_t)(last - i) % C::NS), ((uint32_t)(last - i) / C::NS) & 1, abort_flag, tmo, S_DRAIN, status, false);
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------------ Q producer
        if (lane == 0) {
            int tau = 0;
            for (; walk.next(p.s, g); ++tau) {
                const int i = p.q_bufs == 2 ? tau & 1 : 0, u = p.q_bufs == 2 ? tau >> 1 : tau;   // buffer, its use
                if (u && !bounded_wait(bar_qfree(i), (u - 1) & 1, abort_flag, tmo, S_QFREE, status)) break;
                mbar_arrive_expect_tx(bar_q(i), (uint32_t)(p.q_box * C::PANELS * (PAIR ? 2 : 1)));
                const uint32_t dst = sb + (uint32_t)i * C::PANELS * p.q_panel;
#pragma unroll
                for (int h = 0; h < (PAIR ? 2 : 1); ++h)   // a second tile past the last row is filled with zeros
#pragma unroll
                    for (int pn = 0; pn < C::PANELS; ++pn)
                        tma_load_3d(dst + h * C::QTILE + pn * p.q_panel, &maps.q, pn * 64, g.mt * p.s.tile + h * kRowTile,
                                    g.b * p.s.Hkv + g.kvh, bar_q(i));
            }
            for (int x = max(0, tau - p.q_bufs); x < tau; ++x) {
                const int i = p.q_bufs == 2 ? x & 1 : 0, u = p.q_bufs == 2 ? x >> 1 : x;
                bounded_wait(bar_q(i), u & 1, abort_flag, tmo, S_DRAIN, status, false);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (whole warp)
        constexpr uint32_t idS = idesc_f16(BF16, kRowTile, BN, false), idPV = idesc_f16(BF16, kRowTile, D, true);
        constexpr uint32_t HI = sdesc_hi_sw128(1024);
        Ring<C::NS> ring;
        int tau = 0;
        uint32_t gs = 0;   // this CTA's key step
        uint32_t sQ = sb;
        bool ok = true;
        // S_i = Q K^T with the key tile of ring slot `at`; ready on barS
        auto issue_s = [&](uint32_t i, uint32_t q, uint32_t at) {
            const uint32_t sK = sRing + at * C::KVTILE;
#pragma unroll
            for (int pn = 0; pn < C::PANELS; ++pn)
                mma_ss_kk4_elect(tmem + i * BN, sdesc_lo(q + pn * p.q_panel, 16), sdesc_lo(sK + pn * C::KVPANEL, 16), HI, idS, pn ? 1u : 0u);
            tc_commit_elect(barS + 8u * i);
        };
        // O_acc += P_i V with the value tile of ring slot `at`, 64 keys at a time (all of them, or the half that holds
        // the valid ones); done on barPV
        auto issue_pv = [&](uint32_t i, uint32_t acc, uint32_t at, int valid, bool first) {
            const uint32_t vlo = sdesc_lo(sRing + at * C::KVTILE, C::KVPANEL);
#pragma unroll
            for (int h = 0; h < BN / 64; ++h)
                if (h == 0 || valid > 64)
                    mma_ts_mn4_elect(tmem + C::COL_O + acc * D, tmem + i * BN + 32 * h, vlo + (uint32_t)((h * 8192) >> 4), HI, idPV,
                                     first && h == 0 ? 0u : 1u);
            tc_commit_elect(barPV + 8u * i);
        };
        for (; ok && walk.next(p.s, g); ++tau) {
            const int nk = g.k1 - g.k0;
            const uint32_t qi = p.q_bufs == 2 ? tau & 1 : 0, qu = p.q_bufs == 2 ? tau >> 1 : tau;
            sQ = sb + qi * C::PANELS * p.q_panel;
            ok = wait_all(bar_q(qi), qu & 1, S_Q) && wait_all(bar_full(ring.at), ring.phase, S_FULL);
            if (!ok) break;
            tc_fence_after();
            if constexpr (PAIR) {
                issue_s(0, sQ, ring.at);
                issue_s(1, sQ + C::QTILE, ring.at);
            } else {
                issue_s(gs & 1, sQ, ring.at);
            }
            tc_commit_elect(bar_empty(ring.at));
            if (nk == 1) tc_commit_elect(bar_qfree(qi));
            ring.next();
            for (int j = 0; j < nk; ++j, ++gs) {
                const int valid = valid_of(g, g.k0 + j);
                const bool more = j + 1 < nk;
                uint32_t kat = 0;
                if constexpr (PAIR) {
                    // per step: P V of tile a, its next S, P V of tile b, its next S; an S follows the P V that read its buffer
                    if (more) {
                        ok = wait_all(bar_full(ring.at), ring.phase, S_FULL);
                        if (!ok) break;
                        kat = ring.at;
                        ring.next();
                    }
                    ok = wait_all(bar_full(ring.at), ring.phase, S_FULL);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        ok = ok && wait_all(barP + 8u * i, gs & 1, S_P);
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv(i, i, ring.at, valid, j == 0);
                        if (i == 1) tc_commit_elect(bar_empty(ring.at));
                        if (more) {
                            issue_s(i, sQ + i * C::QTILE, kat);
                            if (i == 1) {
                                tc_commit_elect(bar_empty(kat));
                                if (j + 2 == nk) tc_commit_elect(bar_qfree(qi));
                            }
                        }
                    }
                    if (!ok) break;
                } else {
                    if (more) {
                        ok = wait_all(bar_full(ring.at), ring.phase, S_FULL);
                        if (!ok) break;
                        tc_fence_after();
                        issue_s((gs + 1) & 1, sQ, ring.at);   // its buffer held P(gs - 1), whose P V was issued before
                        tc_commit_elect(bar_empty(ring.at));
                        if (j + 2 == nk) tc_commit_elect(bar_qfree(qi));
                        ring.next();
                    }
                    ok = wait_all(bar_full(ring.at), ring.phase, S_FULL) && wait_all(barP + 8u * (gs & 1), (gs >> 1) & 1, S_P);
                    if (!ok) break;
                    tc_fence_after();
                    issue_pv(gs & 1, NG == 2 ? gs & 1 : 0, ring.at, valid, j < NG);
                    tc_commit_elect(bar_empty(ring.at));
                }
                ring.next();
            }
        }
        tc_commit_elect(barDone);
        bounded_wait(barDone, 0, abort_flag, tmo, S_DRAIN, status, false);
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------------------ softmax, epilogue
        const int grp = (warp - 4) >> 2;
        const int r = (threadIdx.x - 128) & 127;                  // row of the tile == TMEM lane
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const float sl2 = p.sl2;
        const uint64_t sl2x2 = f2_pack(sl2, sl2);
        uint32_t gs0 = 0;
        int use0 = 0, seg = 0;
        bool ok = true;
        // Scores read once, by unrolled code, or twice, by a short loop: the loop where memory is the bound, since what a
        // launch and a unit's end cost is mostly code fetched anew (D = 128: 64 x 512 slots 38 instead of 45 us, 8 x
        // 131072 620 either way), not beside a second row tile, nor at D = 64, where a step is half as long
        // (64 x 1024 slots 41 and 45 us, 64 x 4096 105 and 93, 8 x 131072 351 and 320).
        constexpr bool UNROLLED = PAIR || D == 64;
        const int urow = (PAIR ? grp * kRowTile : 0) + r;          // row of the unit
        for (; ok && walk.next(p.s, g); ++seg) {
            const int nk = g.k1 - g.k0;
            const int row = g.mt * p.s.tile + urow, t = row % p.s.T;
            const bool live = row < p.s.rows && t < g.len.t;
            const bool warp_live = __any_sync(~0u, live);
            const int32_t *parent = p.parent ? p.parent + (size_t)g.b * p.s.T : nullptr;
            float m_used = -INFINITY, l = 0.f;
            bool first = true;
            for (int j = grp >= NG ? nk : PAIR || NG == 1 ? 0 : (int)((gs0 ^ (uint32_t)grp) & 1u); j < nk; j += C::STRIDE) {
                const uint32_t gs = gs0 + j;
                const uint32_t bi = PAIR ? (uint32_t)grp : gs & 1, ph = PAIR ? gs & 1 : (gs >> 1) & 1;   // S buffer, its phase
                const uint32_t tS = tmem + lane_off + bi * BN;
                const int kt = g.k0 + j;
                const bool draft = kt >= g.len.kc;
                const int valid = valid_of(g, kt);
                const bool masked = draft || valid < BN;
                uint32_t bits[BN / 32];
                if (masked) {
                    if (draft && live) {
                        path_bits<BN / 32>(parent, t, (kt - g.len.kc) * BN, bits);
                    } else {
#pragma unroll
                        for (int w = 0; w < BN / 32; ++w) {
                            const int c = valid - 32 * w;
                            bits[w] = c <= 0 || draft ? 0u : (c >= 32 ? ~0u : (1u << c) - 1u);
                        }
                    }
                }
                ok = wait_all(barS + 8u * bi, ph, S_S);
                if (!ok) break;
                tc_fence_after();
                bool rescale = false;
                float alpha = 1.f;
                // the running maximum with this step's: what the sums are relative to, and whether O must follow
                auto grow = [&](float mrow) {
                    const float m_new = fmaxf(m_used, live ? mrow * sl2 : -INFINITY);
                    if (first || m_used == -INFINITY) {
                        // nothing but zeros in this group's O so far
                        m_used = m_new;
                    } else if (m_new - m_used > kTau) {
                        alpha = ex2_approx(m_used - m_new);
                        l *= alpha;
                        m_used = m_new;
                        rescale = true;
                    }
                };
                if (UNROLLED && warp_live && !masked) {
                    uint32_t sv[BN];
                    float pm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < BN; c += 32)
                        tmem_ld_red_max_x32(tS + c, *reinterpret_cast<uint32_t(*)[32]>(sv + c), pm[c / 32]);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < BN; c += 32) reg_fence_x32(*reinterpret_cast<uint32_t(*)[32]>(sv + c));
                    reg_fence_f4(pm[0], pm[1], pm[2], pm[3]);
                    grow(fmaxf(fmax3(pm[0], pm[1], pm[2]), pm[3]));
                    const float *s = reinterpret_cast<const float *>(sv);
                    const float msub = m_used == -INFINITY ? 0.f : m_used;
                    const uint64_t negm2 = f2_pack(-msub, -msub);
                    uint64_t sum2[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum2[i] = f2_pack(0.f, 0.f);
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int i = 32 * c + 2 * e;
                            float t0, t1;
                            f2_unpack(f2_fma(f2_pack(s[i], s[i + 1]), sl2x2, negm2), t0, t1);
                            const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
                            sum2[e & 3] = f2_add(sum2[e & 3], f2_pack(p0, p1));
                            pk[e] = pack2<BF16>(p0, p1);
                        }
                        tmem_st_x16(tS + 16 * c, pk);
                    }
                    float la, lb;
                    f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), la, lb);
                    l += la + lb;
                } else if (warp_live) {
                    // The maximum, then P, 32 keys at a time in a short loop
                    const int chunks = masked ? (valid + 31) >> 5 : BN / 32;
                    uint32_t sv[32];
                    if (masked) {
                        // hidden scores become -inf, up to the last valid one
                        auto word = [&](int c) { return BN == 64 ? (c ? bits[1] : bits[0]) : (c < 2 ? (c ? bits[1] : bits[0]) : (c == 2 ? bits[BN / 32 - 2] : bits[BN / 32 - 1])); };
                        float mrow = -INFINITY;
#pragma unroll 1
                        for (int c = 0; c < chunks; ++c) {
                            tmem_ld_x32(tS + 32 * c, sv);
                            const uint32_t w = word(c);
                            tmem_wait_ld();
                            reg_fence_x32(sv);
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                if (!((w >> e) & 1u)) sv[e] = 0xff800000u;
                                mrow = fmaxf(mrow, __uint_as_float(sv[e]));
                            }
                            tmem_st_x32(tS + 32 * c, sv);
                        }
                        tmem_wait_st();
                        grow(mrow);
                    } else {
                        float pm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int c = 0; c < BN; c += 32) tmem_ld_red_max_x32(tS + c, sv, pm[c / 32]);
                        tmem_wait_ld();
                        reg_fence_f4(pm[0], pm[1], pm[2], pm[3]);
                        grow(fmaxf(fmax3(pm[0], pm[1], pm[2]), pm[3]));
                    }
                    const float msub = m_used == -INFINITY ? 0.f : m_used;
                    const uint64_t negm2 = f2_pack(-msub, -msub);
                    uint64_t sum2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
                    // P of 32 keys overwrites the scores of 16: the scores of later keys are never where it goes
                    tmem_ld_x32(tS, sv);
#pragma unroll 1
                    for (int c = 0; c < chunks; ++c) {
                        tmem_wait_ld();
                        reg_fence_x32(sv);
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float t0, t1;
                            f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), sl2x2, negm2), t0, t1);
                            const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
                            sum2[e & 1] = f2_add(sum2[e & 1], f2_pack(p0, p1));
                            pk[e] = pack2<BF16>(p0, p1);
                        }
                        if (c + 1 < chunks) tmem_ld_x32(tS + 32 * (c + 1), sv);
                        tmem_st_x16(tS + 16 * c, pk);
                    }
                    float la, lb;
                    f2_unpack(f2_add(sum2[0], sum2[1]), la, lb);
                    l += la + lb;
                    if (chunks & 1) {   // P is taken for whole halves of 64 keys
                        const uint32_t none[16] = {};
                        tmem_st_x16(tS + 16 * chunks, none);
                    }
                }
                // O may be rescaled only once this accumulator's previous product is complete
                if (__any_sync(~0u, rescale)) {
                    const uint32_t prev = gs - C::STRIDE;
                    ok = PAIR ? wait_all(barPV + 8u * bi, prev & 1, S_PV) : wait_all(barPV + 8u * (prev & 1), (prev >> 1) & 1, S_PV);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t tO = tmem + lane_off + C::COL_O + (uint32_t)(grp * D);
                    const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t ov[32];
                        tmem_ld_x32(tO + c, ov);
                        tmem_wait_ld();
                        reg_fence_x32(ov);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float lo, hi;
                            f2_unpack(f2_mul(f2_pack(__uint_as_float(ov[e]), __uint_as_float(ov[e + 1])), a2), lo, hi);
                            ov[e] = __float_as_uint(lo);
                            ov[e + 1] = __float_as_uint(hi);
                        }
                        tmem_st_x32(tO + c, ov);
                    }
                }
                if (first && seg > 0) {
                    // every warp is done with the epilogue of the segment before: with both
                    // accumulators, the groups' maxima and sums and the non-finite mark
                    ok = wait_all(barRead, (seg - 1) & 1, S_READ);
                    if (!ok) break;
                }
                if (masked && (!PAIR || grp == 0)) {
                    // V behind the last valid key is zeroed; a drafted V's non-finite values are taken out.  (In a pair
                    // the first group does it: its product is issued before the second's.)
                    const int uv = use0 + (j + 1 < nk ? 2 * j + 2 : 2 * j + 1);
                    ok = wait_all(bar_full(uv % C::NS), (uv / C::NS) & 1, S_FULL);
                    if (!ok) break;
                    const uint32_t sV = sRing + (uint32_t)(uv % C::NS) * C::KVTILE;
                    // 16-byte chunks of one panel; what is behind the last token of all sequences was zeroed when it was loaded
                    const int end = draft ? min(BN, p.s.T - (kt - g.len.kc) * BN) : BN, dead = (min((valid + 63) & ~63, end) - valid) * 8;
#pragma unroll 1
                    for (int pn = 0; pn < C::PANELS; ++pn)
                        for (int i = r; i < dead; i += 128) st_shared_v4(sV + pn * C::KVPANEL + valid * 128 + i * 16, 0u, 0u, 0u, 0u);
                    bool wrote = dead > 0;
                    if (draft) {
                        bool any = false;
#pragma unroll 1
                        for (int pn = 0; pn < C::PANELS; ++pn)
                            for (int i = r; i < valid * 8; i += 128) {
                                const uint32_t a = sV + pn * C::KVPANEL + i * 16;
                                uint32_t w[4];
                                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                             : "r"(a)
                                             : "memory");
                                bool here = false;
#pragma unroll
                                for (int e = 0; e < 4; ++e) w[e] = drop_nonfinite<BF16>(w[e], here);
                                if (here) st_shared_v4(a, w[0], w[1], w[2], w[3]);
                                any |= here;
                            }
                        if (any) misc->nonfinite = seg + 1;
                        wrote |= any;
                    }
                    if (wrote) fence_proxy_async_smem();
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(barP + 8u * bi);
                first = false;
            }
            if (!ok) break;
            // ---- epilogue: join the groups' maxima and sums, then O
            if (first && seg > 0) {   // a segment of one step, the other group's
                ok = wait_all(barRead, (seg - 1) & 1, S_READ);
                if (!ok) break;
            }
            ml[grp * 128 + r] = make_float2(m_used, l);
            __syncwarp();
            if (lane == 0) mbar_arrive(barJoin);
            ok = wait_all(barJoin, seg & 1, S_JOIN);
            if (!ok) break;
            constexpr bool SPLIT = NG == 2 && !PAIR;       // two accumulators of the same rows
            constexpr bool HALF = !PAIR;                   // each group reads half of the columns
            float f0, f1 = 0.f, L = l, M = m_used;
            if constexpr (SPLIT) {
                const float2 a = ml[r], b = ml[128 + r];
                M = fmaxf(a.x, b.x);
                const float ms = M == -INFINITY ? 0.f : M;
                f0 = a.y == 0.f ? 0.f : ex2_approx(a.x - ms);
                f1 = b.y == 0.f ? 0.f : ex2_approx(b.x - ms);
                L = f0 * a.y + f1 * b.y;
                const float inv = L == 0.f ? 0.f : 1.f / L;
                f0 *= inv;
                f1 *= inv;
            } else {
                if constexpr (NG == 1) {
                    L = ml[r].y;
                    M = ml[r].x;
                }
                f0 = L == 0.f ? 0.f : 1.f / L;
            }
            // the last products: this group's, or both groups' (the segment's last two steps, if it has two)
            const uint32_t e1 = gs0 + nk - 1;
            if constexpr (PAIR) {
                ok = wait_all(barPV + 8u * grp, e1 & 1, S_PV);
            } else {
                ok = wait_all(barPV + 8u * (e1 & 1), (e1 >> 1) & 1, S_PV);
                if (ok && nk > 1) ok = wait_all(barPV + 8u * ((e1 - 1) & 1), ((e1 - 1) >> 1) & 1, S_PV);
            }
            if (!ok) break;
            tc_fence_after();
            const bool have0 = !SPLIT || nk > 1 || (gs0 & 1) == 0, have1 = SPLIT && (nk > 1 || (gs0 & 1) == 1);
            const bool whole = g.k0 == 0 && g.k1 == g.len.nt;
            const bool odd = misc->nonfinite == seg + 1;   // rare: non-finite values in the drafted V
            const size_t prow = (size_t)part_slot(blockIdx.x, g.k0) * p.part_rows + urow;
            const size_t orow = ((size_t)(g.b * p.s.Hkv + g.kvh)) * p.s.rows + row;
            constexpr int COLS = HALF ? D / 2 : D;         // columns of this group
            const uint32_t tO0 = tmem + lane_off + C::COL_O + (PAIR ? grp * D : 0);
            if (warp_live) {
                // 16 columns at a time: the code is fetched anew after the key steps, and its length counts more than the loads'
#pragma unroll 1
                for (int c = HALF ? grp * COLS : 0, cn = 0; cn < COLS; c += 16, cn += 16) {
                    uint32_t oa[16], ob[16];
                    tmem_ld_x16(tO0 + c, oa);
                    if constexpr (SPLIT) tmem_ld_x16(tO0 + D + c, ob);
                    tmem_wait_ld();
                    reg_fence_x16(oa);
                    if constexpr (SPLIT) reg_fence_x16(ob);
                    float h[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        // an accumulator without a step holds anything; one with a factor of 0 may hold a non-finite value
                        h[e] = have0 ? __uint_as_float(oa[e]) * f0 : 0.f;
                        if constexpr (SPLIT) h[e] = have1 ? fmaf(__uint_as_float(ob[e]), f1, h[e]) : h[e];
                    }
                    if (live && odd) {
                        // weights are positive, so a non-finite value counts as what it is
                        for (int kt = max(g.k0, g.len.kc); kt < g.k1; ++kt) {
                            const int lo = (kt - g.len.kc) * BN;
                            uint32_t bits[BN / 32];
                            path_bits<BN / 32>(parent, t, lo, bits);
#pragma unroll 1
                            for (int key = lo; key < min(lo + BN, g.len.t); ++key) {
                                uint32_t w = bits[0];
#pragma unroll
                                for (int x = 1; x < BN / 32; ++x) w = (key - lo) >> 5 == x ? bits[x] : w;
                                if (!((w >> ((key - lo) & 31)) & 1u)) continue;
                                const uint16_t *v = static_cast<const uint16_t *>(p.v_new) +
                                                    ((size_t)(g.b * p.s.Hkv + g.kvh) * p.s.T + key) * D + c;
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    const float x = half_to_float<BF16>(v[e]);
                                    if (!isfinite(x)) h[e] += x;
                                }
                            }
                        }
                    }
                    if (live && whole) {
                        uint32_t pk[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) pk[e] = pack2<BF16>(h[2 * e], h[2 * e + 1]);
                        uint8_t *dst = static_cast<uint8_t *>(p.o) + (orow * D + c) * 2;
#pragma unroll
                        for (int q4 = 0; q4 < 2; ++q4)
                            st_global_v4(dst + q4 * 16, pk[4 * q4], pk[4 * q4 + 1], pk[4 * q4 + 2], pk[4 * q4 + 3]);
                    } else if (live) {
                        float *dst = p.part_o + prow * D + c;
#pragma unroll
                        for (int q8 = 0; q8 < 2; ++q8) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(h[8 * q8 + e]);
                            st_global_v8(dst + 8 * q8, w);
                        }
                    }
                    __syncwarp();   // the next columns are read by all lanes together
                }
            }
            if (live && (!HALF || grp == 0)) {
                const float lse2 = L == 0.f ? -INFINITY : M + lg2_approx(L);
                if (whole)
                    p.lse[orow] = lse2 * 0.69314718055994531f;
                else
                    p.part_lse[prow] = lse2;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(barRead);
            gs0 += nk;
            use0 += 2 * nk;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    } else if (warp >= 4 && *abort_flag) {
        leave_nan<D>(p, const_cast<const Misc *>(misc)->share, threadIdx.x - 128, 256);   // this CTA gave up on a wait
    }
}

// Joins the parts of the units that a cut crosses: o = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M).
// Block x looks whether CTA x + 1 left such a unit (the unit's first cut is the start of its share).  A row in
// a few parts takes one warp; one in many parts (a sequence over the whole GPU) all four, every fourth part
// each.  The parts are added in the same order on every run.
constexpr int kJoinWarps = 4;

template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ TreeParams p)
{
    constexpr int PER = D / 32, FEW = 5;
    __shared__ float sums[kJoinWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_wait();
    grid_done_soon();
    const Cut c = p.cuts[blockIdx.x + 1];
    const int parts = c.parts;
    if (parts == 0) return;
    const int wide = parts > 2 * FEW ? kJoinWarps : 1;            // warps of a row
    const int sub = wide > 1 ? warp : 0, rows = kJoinWarps / wide;
    for (int r0 = blockIdx.y * rows; r0 < p.part_rows; r0 += gridDim.y * rows) {
        const int r = r0 + (wide > 1 ? 0 : warp), row = c.tile * p.s.tile + r;
        const bool live = r < p.part_rows && row < p.s.rows && row % p.s.T < c.n;
        auto prow = [&](int i) { return (size_t)part_slot((int)blockIdx.x + i, i) * p.part_rows + r; };
        float acc[PER], sum = 0.f, M = -INFINITY;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] = 0.f;
        if (live) {
            // the first rows are on their way while the weights (every warp: of all parts) are worked out
            float x[FEW][PER];
            auto fetch = [&](int i0) {
#pragma unroll
                for (int j = 0; j < FEW; ++j)
#pragma unroll
                    for (int e = 0; e < PER; e += 2) {
                        const int i = i0 + j * wide;
                        const float2 v = i < parts ? *reinterpret_cast<const float2 *>(p.part_o + prow(i) * D + lane * PER + e) : make_float2(0.f, 0.f);
                        x[j][e] = v.x;
                        x[j][e + 1] = v.y;
                    }
            };
            const float mine = lane < parts ? p.part_lse[prow(lane)] : -INFINITY;
            fetch(sub);
            M = mine;
            for (int i = lane + 32; i < parts; i += 32) M = fmaxf(M, p.part_lse[prow(i)]);
#pragma unroll
            for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, d));
            const float ms = M == -INFINITY ? 0.f : M;
            const float w = lane < parts ? ex2_approx(mine - ms) : 0.f;
            sum = w;
            for (int i = lane + 32; i < parts; i += 32) sum += ex2_approx(p.part_lse[prow(i)] - ms);
#pragma unroll
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
#pragma unroll 1
            for (int i0 = sub; i0 < parts; i0 += FEW * wide) {
                if (i0 != sub) fetch(i0);
#pragma unroll
                for (int j = 0; j < FEW; ++j) {
                    const int i = i0 + j * wide;
                    if (i >= parts) break;
                    const float f = i < 32 ? __shfl_sync(~0u, w, i & 31) : ex2_approx(p.part_lse[prow(i)] - ms);
#pragma unroll
                    for (int e = 0; e < PER; ++e) acc[e] = fmaf(f, x[j][e], acc[e]);
                }
            }
        }
        if (wide > 1) {
#pragma unroll
            for (int e = 0; e < PER; ++e) sums[warp][lane * PER + e] = acc[e];
            __syncthreads();
            if (sub == 0)
#pragma unroll
                for (int x = 1; x < kJoinWarps; ++x)
#pragma unroll
                    for (int e = 0; e < PER; ++e) acc[e] += sums[x][lane * PER + e];
            __syncthreads();
        }
        if (live && sub == 0) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const size_t orow = (size_t)(c.b * p.s.Hkv + c.kvh) * p.s.rows + row;
            uint32_t *dst = static_cast<uint32_t *>(p.o) + (orow * D + lane * PER) / 2;
#pragma unroll
            for (int e = 0; e < PER / 2; ++e) dst[e] = pack2<BF16>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
            if (lane == 0) p.lse[orow] = sum == 0.f ? -INFINITY : (M + lg2_approx(sum)) * 0.69314718055994531f;
        }
    }
}

template <int D, bool BF16, bool PAIR>
cudaError_t launch_one(const TreeMaps &m, const TreeParams &p0, cudaStream_t st)
{
    using C = Cfg<D, PAIR>;
    auto kern = tree_kernel<D, BF16, PAIR>;
    static std::atomic<uint64_t> configured{0};
    static std::atomic<int> sm_count[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const uint64_t bit = 1ull << dev;
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::ALLOC);
        if (e != cudaSuccess) return e;
        int nsm = 0;
        e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        sm_count[dev].store(nsm, std::memory_order_relaxed);
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    TreeParams p = p0;
    if (p.timeout_ns == 0) p.timeout_ns = kDefaultTimeoutNs;
    const int grid = clampi(sm_count[dev].load(std::memory_order_relaxed), 1, kMaxCtas);
    e = launch_overlapped(kern, dim3(grid), C::THREADS, C::ALLOC, 1, st, m, p);
    if (e != cudaSuccess || grid == 1) return e;
    return launch_overlapped(join_kernel<D, BF16>, dim3(grid - 1, clampi(p.part_rows, 1, 32)), 32 * kJoinWarps, 0, 1, st, p);
}

} // namespace

int tree_log_keys(int D) { return D == 256 ? 6 : 7; }

int tree_tile(int D, long long rows) { return rows > kRowTile && D != 256 ? 2 * kRowTile : kRowTile; }

cudaError_t launch_tree(int D, bool bf16, const TreeMaps &m, const TreeParams &p, cudaStream_t st)
{
    const bool pair = p.s.tile > kRowTile;
#define TREE_CASE(DD, BB, PP) \
    if (D == DD && bf16 == BB && pair == PP) return launch_one<DD, BB, PP>(m, p, st);
    TREE_CASE(64, true, false) TREE_CASE(64, true, true) TREE_CASE(64, false, false) TREE_CASE(64, false, true)
    TREE_CASE(128, true, false) TREE_CASE(128, true, true) TREE_CASE(128, false, false) TREE_CASE(128, false, true)
    TREE_CASE(256, true, false) TREE_CASE(256, false, false)
#undef TREE_CASE
    return cudaErrorInvalidValue;
}

cudaError_t read_and_clear_tree_status(uint32_t *word)
{
    unsigned int w = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&w, g_tree_status, sizeof(w));
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_tree_status, &zero, sizeof(zero));
    if (word) *word = w;
    return e;
}

} // namespace cache
} // namespace fa
