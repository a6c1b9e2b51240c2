// weigh_sm103.cu -- the attention weight that the slots of a cache have received (fa_cache_weights).
//
// For sequence b, KV head c and slot j of its n_b:
//
//     out[b, c, j] = weight[b, c, j] + sum_{h in c} sum_{i < count[b]} [j visible to i] exp(scale q_hi.k_j - lse_hi)
//
// where row i is the query of slot n_b - count[b] + i and, with the causal mask, sees the slots up to its
// own.  The attention that made lse has left the probabilities behind, so one pass over Q K^T suffices:
// no running maximum, no second product.
//
// The score tile is computed transposed, S^T = K Q^T: the keys are the 128 lanes of tensor memory and
// the query rows its columns, so the sum over rows runs along the registers of one thread and no lanes
// are joined.  One packed FMA, one exponential and one packed add a score: a long prompt is bound by the
// tensor pipe and by the exponentials about equally (128 x 128 scores: 512 cycles of each at D = 128),
// a drafting step by the one read of K.
//
// Measured, 32 heads over 8 KV heads, bf16:
//     16 rows a head over 4 x 131072 slots    D = 64 5.9 TB/s (96 us; 16-slot pages 4.3), D = 128 6.5 (170 us; 6.3),
//                                             D = 256 6.8 (319 us; 6.6); one token over 64 x 1024 slots 4.5 (31 us)
//     a prompt over itself, causal            8192 tokens: D = 64 203 us, D = 128 208 us (1320 TFLOP/s), D = 256
//                                             340 us (1620); 2048 tokens, D = 128: 26 us; 16384: 770 us (1430) in
//                                             bursts, 830 to 850 when repeated for seconds (power limit, 1.9 GHz)
//     few rows over a short cache             8 to 10 us: start, one tile, second kernel
// D = 64 has as many exponentials as D = 128 for half the products, and is bound by them.
//
// The steps (key tile x tile of query rows) are shared out evenly (cache_schedule.h).  A key tile that a
// cut crosses leaves its parts in the workspace; a second kernel adds them in order, so the sums do
// not vary from run to run.
//
// Per CTA (one per SM):
//   warps 0, 20   K producers, alternate key tiles (one box per page and panel; one warp for all: D = 64 4.9 TB/s,
//                 D = 128 6.4, with 16-slot pages 3.2 and 4.7); warp 0 is the Q producer too, unless rows are gathered
//   warp 1        TMEM owner and MMA issuer, into four S^T buffers
//   warps 2-3     lse and visible limit of each step's 128 rows; in path mode also the gathered Q tile
//   warps 4-19    the sums, one thread per key: four groups of four warps take the steps in turn, a
//                 buffer each, and are joined at the end of a key tile
// A K or Q tile stays where it is while consecutive steps use it.
#include <atomic>
#include <cstdint>

#include "cache_device.cuh"
#include "cache_internal.h"
#include "ptx.cuh"
#include "watchdog.cuh"

namespace fa {

__device__ unsigned int g_weigh_status;

namespace cache {

namespace {

constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;
constexpr int NB = 4;   // S^T buffers, 128 columns apart, each with a group of four warps that sums it
constexpr int THREADS = 128 + 128 * NB + 32;

enum Site : uint32_t { S_KEMPTY = 1, S_QEMPTY = 2, S_KFULL = 3, S_QFULL = 4, S_FREE = 5, S_S = 6, S_ROWS = 7, S_DRAIN = 8, S_JOIN = 10, S_READ = 11 };

template <int D>
struct Cfg {
    static constexpr int NQ = D == 256 ? 64 : 128;     // query rows of a step
    static constexpr int PANELS = D / 64;
    static constexpr int KPANEL = 128 * 128, KTILE = PANELS * KPANEL;
    static constexpr int QPANEL = NQ * 128, QTILE = PANELS * QPANEL;
    static constexpr int KS = D == 256 ? 2 : (D == 128 ? 4 : 8), QS = 2;   // K is streamed, Q changes now and then
    static constexpr int OFF_Q = KS * KTILE;
    static constexpr int OFF_BAR = OFF_Q + QS * QTILE;
    static constexpr int NBAR = 2 * KS + 2 * QS + 3 * NB + 2 * NB + 1;   // K, Q (full, empty); S, rows, free; join, read; done
    static constexpr int OFF_ROWS = OFF_BAR + ((NBAR * 8 + 15) / 16) * 16;   // NB x { lse2[128], limit[128] }
    static constexpr int OFF_JOIN = OFF_ROWS + NB * 1024;                    // [NB][128] sums handed over
    static constexpr int OFF_MISC = OFF_JOIN + NB * 512;
    static constexpr int BYTES = OFF_MISC + 128;
    static constexpr int ALLOC = BYTES + 1024;   // the base is aligned to 1024 bytes, wherever it is
    static_assert(ALLOC <= 232448, "shared memory of one CTA");
};

struct Misc {
    uint32_t tmem;
    int abort;
    int lowest[NB], cols[NB];   // of each step in flight: lowest limit of its rows, how many rows
    WeighWalk share;            // this CTA's share, not walked yet
};

template <int D, bool BF16>
__global__ void __launch_bounds__(THREADS, 1)
    weigh_kernel(const __grid_constant__ WeighMaps maps, const __grid_constant__ WeighParams p)
{
    using C = Cfg<D>;
    constexpr int NQ = C::NQ;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sb = raw + pad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sQ = sb + C::OFF_Q, bar0 = sb + C::OFF_BAR;
    auto k_full = [&](uint32_t i) { return bar0 + 8u * i; };
    auto k_empty = [&](uint32_t i) { return bar0 + 8u * (C::KS + i); };
    const uint32_t barQ0 = bar0 + 16u * C::KS;
    auto q_full = [&](uint32_t i) { return barQ0 + 8u * i; };
    auto q_empty = [&](uint32_t i) { return barQ0 + 8u * (C::QS + i); };
    const uint32_t barS = barQ0 + 16u * C::QS, barRows = barS + 8u * NB, barFree = barRows + 8u * NB, barJoin = barFree + 8u * NB,
                   barRead = barJoin + 8u * NB, barDone = barRead + 8u * NB;
    float *rows_lse = reinterpret_cast<float *>(smem + C::OFF_ROWS);
    float *join = reinterpret_cast<float *>(smem + C::OFF_JOIN);
    volatile Misc *misc = reinterpret_cast<volatile Misc *>(smem + C::OFF_MISC);
    volatile int *abort_flag = &misc->abort;
    unsigned int *status = &g_weigh_status;
    const uint64_t tmo = p.timeout_ns;
    const bool gather = p.s.mode == kPath;

    grid_done_soon();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::KS; ++s) {
            mbar_init(k_full(s), 1);
            mbar_init(k_empty(s), 1);
        }
        for (int s = 0; s < C::QS; ++s) {
            mbar_init(q_full(s), gather ? 2 : 1);
            mbar_init(q_empty(s), 1);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(barS + 8 * i, 1);
            mbar_init(barRows + 8 * i, 1);
            mbar_init(barFree + 8 * i, 4);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(barJoin + 8 * i, 4);
            mbar_init(barRead + 8 * i, 4);
        }
        mbar_init(barDone, 1);
        misc->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(const_cast<uint32_t *>(&misc->tmem)), 512);
        tmem_relinquish();
    }
    int total = 0, ctas = 1;   // (warp 3) all steps, the CTAs that share them
    if (warp == 3) {
        grid_wait();
        const Share w = find_share(p.s.B, lane, blockIdx.x, gridDim.x, [&](int b) {
            const WeighLen l = weigh_len(p.s, b);
            return p.s.Hkv * weigh_before(l, l.kt);
        });
        const WeighWalk mine(p.s, w.b, w.off, w.left);
        total = w.total;
        ctas = w.G;
        if (lane == 0) const_cast<Misc *>(misc)->share = mine;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_wait();   // every thread: what it reads and writes from here on may be the kernel's before
    const uint32_t tmem = misc->tmem;
    WeighWalk walk = const_cast<const Misc *>(misc)->share;
    WeighRun g;
    const WarpWait wait_all{abort_flag, tmo, status};
    // A Q tile is taken anew with every head, and with every step where a key tile has several: then the
    // tiles 0 .. ns - 1 follow one another again and again.

    if (warp == 0 || warp == 4 + 4 * NB) {
        // ------------------------------------------------------------ K producers, Q producer
        const int who = warp == 0 ? 0 : 1;   // this warp's key tiles: every other one
        const int boxes = div2(128, p.box_rows);
        int ku = 0, qu = 0;
        int skip = -1;   // the key tile that a fault injection leaves out
        const bool inject = who == 0 && ((p.inject & 1u) || ((p.inject & 2u) && blockIdx.x == 0));
        Ring<C::KS> k;
        Ring<C::QS> q;
        bool ok = true;
        while (ok && walk.next_run(p.s, g)) {
            const int units = (g.s + g.steps + g.ns - 1) / g.ns;
            PageRun run;
            bool start = true;
            int step = 0;      // steps whose Q tile has been loaded
            for (int u = 0; ok && u < units; ++u, ++ku, k.next()) {
                const int kt = g.kt + u;
                run.at(p.pages, p.box_rows, g.b, g.len.n, kt * boxes, (g.kt + units) * boxes, lane, start);
                start = false;
                if (((ku ^ who) & 1) == 0) {
                    ok = wait_all(k_empty(k.at), k.phase ^ 1, S_KEMPTY);
                    if (!ok) break;
                    const int valid = min(boxes, cdiv2(g.len.n - kt * 128, p.box_rows));
                    if (skip >= 0 || !inject) {
                        if (lane == 0) mbar_arrive_expect_tx(k_full(k.at), (uint32_t)(valid * p.box_rows * 128 * C::PANELS));
                        __syncwarp();
                        load_boxes<C::PANELS>(sb + k.at * C::KTILE, C::KPANEL, p.box_rows * 128, &maps.k, g.kvh, run.page, run.row, kt * boxes & 31,
                                              valid, k_full(k.at));
                    } else {
                        skip = ku;
                    }
                }
                if (gather || who) continue;
                const int last = min(g.steps, (u + 1) * g.ns - g.s);   // steps up to the end of this key tile
                for (; ok && step < last; ++step) {
                    if (g.ns == 1 && step > 0) continue;
                    ok = wait_all(q_empty(q.at), q.phase ^ 1, S_QEMPTY);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(q_full(q.at), C::QTILE);
#pragma unroll
                        for (int pq = 0; pq < C::PANELS; ++pq)
                            tma_load_3d(sQ + q.at * C::QTILE + pq * C::QPANEL, &maps.q, pq * 64, (g.s + step) % g.ns * NQ, g.b * p.s.Hkv + g.kvh,
                                        q_full(q.at));
                    }
                    ++qu;
                    q.next();
                }
            }
        }
        if (lane == 0) {
            for (int x = max(0, ku - C::KS); x < ku; ++x)
                if (x != skip && ((x ^ who) & 1) == 0) bounded_wait(k_full(x % C::KS), (x / C::KS) & 1, abort_flag, tmo, S_DRAIN, status, false);
            for (int x = max(0, qu - C::QS); x < qu; ++x) bounded_wait(q_full(x % C::QS), (x / C::QS) & 1, abort_flag, tmo, S_DRAIN, status, false);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (whole warp)
        constexpr uint32_t HI = sdesc_hi_sw128(1024);
        Ring<C::KS> k;                       // the next K tile, the next Q tile
        Ring<C::QS> q;
        Ring<NB> st;                         // the step's buffer
        uint32_t k_old = 0, q_old = 0;       // tiles in use, and whether there are any to give back
        bool k_held = false, q_held = false, ok = true;
        while (ok && walk.next_run(p.s, g)) {
            int s = g.s;                     // step of the key tile
            for (int i = 0; i < g.steps; ++i, st.next()) {
                if (i == 0 || s == 0) {
                    if (k_held) tc_commit_elect(k_empty(k_old));   // the last key tile's products are all issued
                    ok = wait_all(k_full(k.at), k.phase, S_KFULL);
                    if (!ok) break;
                    k_old = k.at;
                    k_held = true;
                    k.next();
                }
                if (i == 0 || g.ns > 1) {
                    if (q_held) tc_commit_elect(q_empty(q_old));
                    ok = wait_all(q_full(q.at), q.phase, S_QFULL);
                    if (!ok) break;
                    q_old = q.at;
                    q_held = true;
                    q.next();
                }
                ok = wait_all(barFree + 8u * st.at, st.phase ^ 1, S_FREE);
                if (!ok) break;
                tc_fence_after();
                // columns: the rows of this tile, to the next multiple of 16
                const int cols = max(16, min(NQ, (g.len.rows - s * NQ + 15) & ~15));
                const uint32_t id = idesc_f16(BF16, 128, 16, false) + ((uint32_t)(cols - 16) >> 3 << 17);
                const uint32_t sK = sb + k_old * C::KTILE, sq = sQ + q_old * C::QTILE;
#pragma unroll
                for (int pn = 0; pn < C::PANELS; ++pn)
                    mma_ss_kk4_elect(tmem + st.at * 128u, sdesc_lo(sK + pn * C::KPANEL, 16), sdesc_lo(sq + pn * C::QPANEL, 16), HI, id,
                                     pn ? 1u : 0u);
                tc_commit_elect(barS + 8u * st.at);
                if (g.ns > 1) {   // the next step has another Q tile
                    tc_commit_elect(q_empty(q_old));
                    q_held = false;
                }
                if (++s == g.ns) s = 0;
            }
        }
        tc_commit_elect(barDone);
        bounded_wait(barDone, 0, abort_flag, tmo, S_DRAIN, status, false);
        __syncwarp();
    } else if (warp < 4) {
        // ------------------------------------------------------------ rows: lse, limits, gathered queries
        // The two warps take alternate steps, a lane four neighbouring rows; what a tile's rows need is
        // looked up once while consecutive steps use it.
        if (warp == 3 && lane == 0) {   // for the joining kernel
            Cut c = {};
            if (walk.left > 0) c = Cut{walk.b, walk.kvh, walk.kt, parts_from(total, ctas, blockIdx.x, walk.s, weigh_steps(walk.len, walk.kt)), walk.len.n, {}};
            p.cuts[blockIdx.x] = c;
        }
        const int half = warp - 2;
        Ring<C::QS> q;
        Ring<NB> st;
        bool ok = true;
        while (ok && walk.next_run(p.s, g)) {
            const size_t head0 = (size_t)(g.b * p.s.Hkv + g.kvh) * p.s.group;   // first query head of the group
            const int32_t *path = p.path + (gather ? (size_t)g.b * p.s.T : 0);
            float neg[4] = {0.f, 0.f, 0.f, 0.f};      // -lse, log2 units
            int limit[4] = {0, 0, 0, 0}, low = 0, cols = 0;
            bool fresh = true;
            int s = g.s;
            for (int i = 0; i < g.steps; ++i, st.next(), s = s + 1 == g.ns ? 0 : s + 1) {
                const int row0 = s * NQ;
                if (gather && (i == 0 || g.ns > 1)) {
                    ok = wait_all(q_empty(q.at), q.phase ^ 1, S_QEMPTY);
                    if (!ok) break;
                    const uint32_t dst = sQ + q.at * C::QTILE;
                    // rows to the next multiple of 16; 16-byte chunk c of row r at c ^ (r & 7) of its 128 bytes
                    const int rows = min(NQ, max(16, (g.len.rows - row0 + 15) & ~15));
                    // (four of a thread's chunks are read before the first is stored)
                    const int all = rows * (D / 8);
                    for (int x0 = threadIdx.x - 64; x0 < all; x0 += 4 * 64) {
                        uint4 v[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int x = x0 + 64 * u, row = row0 + x / (D / 8);
                            v[u] = make_uint4(0, 0, 0, 0);
                            if (x < all && row < g.len.rows) {
                                const int h = row / g.len.a, t = path[row - h * g.len.a];
                                if (t >= 0 && t < p.s.T) v[u] = static_cast<const uint4 *>(p.q)[((head0 + h) * p.s.T + t) * (D / 8) + x % (D / 8)];
                            }
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int x = x0 + 64 * u, r = x / (D / 8), ch = x % (D / 8);
                            if (x < all) st_shared_v4(dst + (ch >> 3) * C::QPANEL + r * 128 + (((ch & 7) ^ (r & 7)) << 4), v[u].x, v[u].y, v[u].z, v[u].w);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(q_full(q.at));
                    q.next();
                }
                if ((int)(st.at & 1) != half) continue;
                if (fresh || g.ns > 1) {
                    fresh = false;
                    low = 0x7fffffff;
                    cols = min(NQ, g.len.rows - row0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = 4 * lane + e, row = row0 + c;
                        int order = -1, h = 0, t = 0;      // order of the row, its head in the group, its place in q
                        if (c < cols) {
                            const int len = gather ? g.len.a : p.s.T;
                            h = row / len;
                            order = t = row - h * len;
                            if (gather) t = path[order];
                            if (order >= g.len.a || t < 0 || t >= p.s.T) order = -1;
                        }
                        limit[e] = 0;
                        neg[e] = 0.f;
                        if (order >= 0) {
                            const float v = p.lse[(head0 + h) * p.s.T + t];
                            neg[e] = v * -1.4426950408889634f;
                            // a row that saw nothing gave nothing
                            limit[e] = v == -INFINITY ? 0 : (p.s.causal ? clampi(g.len.off + order + 1, 0, g.len.n) : g.len.n);
                        }
                        if (c < NQ) low = min(low, limit[e]);
                    }
                    low = __reduce_min_sync(~0u, low);
                }
                ok = wait_all(barFree + 8u * st.at, st.phase ^ 1, S_FREE);
                if (!ok) break;
                reinterpret_cast<float4 *>(rows_lse + st.at * 256)[lane] = make_float4(neg[0], neg[1], neg[2], neg[3]);
                reinterpret_cast<int4 *>(rows_lse + st.at * 256 + 128)[lane] = make_int4(limit[0], limit[1], limit[2], limit[3]);
                if (lane == 0) {
                    misc->lowest[st.at] = low;
                    misc->cols[st.at] = cols;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(barRows + 8u * st.at);
            }
        }
    } else {
        // ------------------------------------------------------------ sums, one thread per key
        const int grp = (warp - 4) >> 2, r = (threadIdx.x - 128) & 127;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint64_t sl2x2 = f2_pack(p.sl2, p.sl2);
        uint32_t st0 = 0;     // steps before
        uint32_t posts = 0;   // parity of the sums that each group has handed over (bit), that it has any (bit + NB)
        bool ok = true;
        // what this key receives in step `st` (this group's: buffer grp)
        auto receive = [&](uint32_t st, int key0, float &sum) -> bool {
            const uint32_t bi = grp, ph = (st / NB) & 1;
            const int slot = key0 + r;
            if (!wait_all(barRows + 8u * bi, ph, S_ROWS) || !wait_all(barS + 8u * bi, ph, S_S)) return false;
            tc_fence_after();
            const float *neg = rows_lse + bi * 256;
            const int *limit = reinterpret_cast<const int *>(neg) + 128;
            const uint32_t tS = tmem + lane_off + bi * 128u;
            const int cols = misc->cols[bi];
            uint64_t sum2[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) sum2[i] = f2_pack(0.f, 0.f);
            // 32 columns: exp2(s sl2 - lse2), two columns to an instruction but for the exponential
            auto add = [&](const uint32_t(&sv)[32], int c, bool masked) {
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const ulonglong2 l = *reinterpret_cast<const ulonglong2 *>(neg + c + e);
                    float x[4];
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), sl2x2, l.x), x[0], x[1]);
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[e + 2]), __uint_as_float(sv[e + 3])), sl2x2, l.y), x[2], x[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = ex2_approx(x[i]);
                    if (masked) {
                        const int4 m = *reinterpret_cast<const int4 *>(limit + c + e);
                        x[0] = slot < m.x ? x[0] : 0.f;
                        x[1] = slot < m.y ? x[1] : 0.f;
                        x[2] = slot < m.z ? x[2] : 0.f;
                        x[3] = slot < m.w ? x[3] : 0.f;
                    }
                    sum2[(e >> 1) & 3] = f2_add(sum2[(e >> 1) & 3], f2_pack(x[0], x[1]));
                    sum2[((e >> 1) + 1) & 3] = f2_add(sum2[((e >> 1) + 1) & 3], f2_pack(x[2], x[3]));
                }
            };
            const bool masked = misc->lowest[bi] < key0 + 128;   // some row does not see the whole key tile
#pragma unroll 1
            for (int c = 0; c < cols; c += 32) {
                uint32_t sv[32];
                tmem_ld_x32(tS + c, sv);
                tmem_wait_ld();
                reg_fence_x32(sv);
                if (masked)
                    add(sv, c, true);
                else
                    add(sv, c, false);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(barFree + 8u * bi);
            float la, lb;
            f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), la, lb);
            sum += la + lb;
            return true;
        };
        while (ok && walk.next_run(p.s, g)) {
            const size_t head = (size_t)(g.b * p.s.Hkv + g.kvh) * p.s.capacity;
            if (g.ns == 1) {
                // a step is a key tile, and no other group has a part in it
                for (int i = (int)(((uint32_t)grp - st0) % NB); i < g.steps; i += NB) {
                    const int key0 = (g.kt + i) * 128, slot = key0 + r;
                    const bool live = slot < g.len.n;
                    float sum = 0.f;
                    const float base = live && p.weight ? p.weight[head + slot] : 0.f;
                    ok = receive(st0 + i, key0, sum);
                    if (!ok) break;
                    if (live) p.out[head + slot] = base + sum;
                }
                st0 += g.steps;
                continue;
            }
            int done = 0;
            for (int kt = g.kt, s0 = g.s; ok && done < g.steps; ++kt, s0 = 0) {
                const int ns = min(g.steps - done, g.ns - s0);           // this CTA's steps of the key tile
                const int key0 = kt * 128, slot = key0 + r;
                const bool whole = ns == g.ns, live = slot < g.len.n;
                const int owner = (int)((st0 + ns - 1) % NB);            // the group of the last step
                float base = 0.f, sum = 0.f;
                if (grp == owner && whole && live && p.weight) base = p.weight[head + slot];
                for (int i = (int)(((uint32_t)grp - st0) % NB); ok && i < ns; i += NB) ok = receive(st0 + i, key0, sum);
                if (!ok) break;
                // the other groups of the key tile hand their sums to the owner of its last step, which adds
                // them in the order of their steps
                for (int x = ns < NB ? ns - 1 : NB - 1; ok && x > 0; --x) {
                    const int other = (owner - x + NB) % NB;
                    const uint32_t par = (posts >> other) & 1u, any = (posts >> (NB + other)) & 1u;
                    posts = (posts ^ (1u << other)) | (1u << (NB + other));
                    if (grp == other) {
                        if (any) ok = wait_all(barRead + 8u * other, par ^ 1u, S_READ);
                        if (!ok) break;
                        join[other * 128 + r] = sum;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(barJoin + 8u * other);
                    } else if (grp == owner) {
                        ok = wait_all(barJoin + 8u * other, par, S_JOIN);
                        if (!ok) break;
                        sum += join[other * 128 + r];
                        __syncwarp();
                        if (lane == 0) mbar_arrive(barRead + 8u * other);
                    }
                }
                if (!ok) break;
                if (grp == owner && live) {
                    if (whole)
                        p.out[head + slot] = base + sum;
                    else
                        p.part[(size_t)part_slot(blockIdx.x, s0) * 256 + r] = sum;
                }
                st0 += ns;
                done += ns;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    } else if (warp >= 4 && warp < 8 && *abort_flag) {
        // This CTA gave up on a wait: NaN into every sum it was given
        const int r = threadIdx.x - 128;
        walk = const_cast<const Misc *>(misc)->share;
        WeighSeg g;
        while (walk.next(p.s, g)) {
            if (g.kt * 128 + r >= g.len.n) continue;
            if (g.s0 == 0 && g.s1 == g.ns)
                p.out[(size_t)(g.b * p.s.Hkv + g.kvh) * p.s.capacity + g.kt * 128 + r] = __uint_as_float(~0u);
            else
                p.part[(size_t)part_slot(blockIdx.x, g.s0) * 256 + r] = __uint_as_float(~0u);
        }
    }
}

// ---------------------------------------------------------------- long prompts
// Every query row against every earlier slot: bound by the tensor pipe and the exponentials, if the
// operands keep up.  With K and Q both in shared memory the products alone read 64 KB of it per 128 x 128
// scores at D = 128, all that it delivers in the 512 cycles of the products, and each Q tile is fetched for
// one key tile only.  So a unit is two key tiles, copied into tensor memory once and used as the A operand
// (lanes = keys), and each Q tile is multiplied with both: 48 KB of shared-memory traffic per 128 x 128
// scores, the Q tile's own arrival included.
//   tensor memory   K_0, K_1 (D / 2 columns each), then NBUF score buffers of NQ columns
//   warps 0, 1, 2-3 as above;  warps 4-7 and 8-11 the sums of the first and the second key tile
template <int D>
struct Prompt {
    static constexpr int THREADS = 384;
    static constexpr int NQ = D == 256 ? 64 : 128;
    static constexpr int NBUF = D == 256 ? 4 : 3;     // score buffers
    static constexpr int NR = 4;                       // steps whose rows are looked up ahead
    static constexpr int PANELS = D / 64;
    static constexpr int KPANEL = 256 * 128, KPAIR = PANELS * KPANEL;   // both key tiles, 256 rows to a panel
    static constexpr int QPANEL = NQ * 128, QTILE = PANELS * QPANEL;
    static constexpr int QS = D == 256 ? 2 : (D == 128 ? 4 : 8);
    static constexpr int OFF_Q = KPAIR;
    static constexpr int OFF_BAR = OFF_Q + QS * QTILE;
    static constexpr int NBAR = 2 + 2 * QS + 2 * NBUF + 2 * NR + 2;     // K, Q (full, empty); S (full, free); rows (full, free); unit, done
    static constexpr int OFF_ROWS = OFF_BAR + ((NBAR * 8 + 15) / 16) * 16;   // NR x { -lse2[128], limit[128] }
    static constexpr int OFF_MISC = OFF_ROWS + NR * 1024;
    static constexpr int BYTES = OFF_MISC + 128;
    static constexpr int ALLOC = BYTES + 1024;   // the base is aligned to 1024 bytes, wherever it is
    static_assert(ALLOC <= 232448, "shared memory of one CTA");
    static constexpr uint32_t COL_S = D;               // the scores start behind the two key tiles
    static_assert(D + NBUF * NQ <= 512, "tensor-memory columns");
};

// One 64-column panel of 128 rows, 128-byte swizzled, into 32 tensor-memory columns (lane = row).
__device__ __forceinline__ void copy_panel_elect(uint32_t t, uint32_t lo, uint32_t hi)
{
    asm volatile("{\n\t.reg .b32 ta, al;\n\t.reg .b64 a;\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "mov.b64 a, {%1, %2};\n\t@e tcgen05.cp.cta_group::1.128x256b [%0], a;\n\t"
                 "add.u32 ta, %0, 8;\n\tadd.u32 al, %1, 2;\n\tmov.b64 a, {al, %2};\n\t@e tcgen05.cp.cta_group::1.128x256b [ta], a;\n\t"
                 "add.u32 ta, %0, 16;\n\tadd.u32 al, %1, 4;\n\tmov.b64 a, {al, %2};\n\t@e tcgen05.cp.cta_group::1.128x256b [ta], a;\n\t"
                 "add.u32 ta, %0, 24;\n\tadd.u32 al, %1, 6;\n\tmov.b64 a, {al, %2};\n\t@e tcgen05.cp.cta_group::1.128x256b [ta], a;\n\t}"
                 ::"r"(t), "r"(lo), "r"(hi)
                 : "memory");
}

// Four K-steps of D(tmem) (+)= A(tmem) B(smem, K-major).
__device__ __forceinline__ void mma_ts_k4_elect(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .b32 ta, bl;\n\t.reg .b64 b;\n\t.reg .pred p, e, t;\n\t"
                 "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "mov.b64 b, {%2, %3};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t"
                 "add.u32 ta, %1, 8;\n\tadd.u32 bl, %2, 2;\n\tmov.b64 b, {bl, %3};\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], b, %4, t;\n\t"
                 "add.u32 ta, %1, 16;\n\tadd.u32 bl, %2, 4;\n\tmov.b64 b, {bl, %3};\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], b, %4, t;\n\t"
                 "add.u32 ta, %1, 24;\n\tadd.u32 bl, %2, 6;\n\tmov.b64 b, {bl, %3};\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], b, %4, t;\n\t}"
                 ::"r"(d), "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
                 : "memory");
}

template <int D, bool BF16, bool LONG>
__global__ void __launch_bounds__(Prompt<D>::THREADS, 1)
    weigh_prompt_kernel(const __grid_constant__ WeighMaps maps, const __grid_constant__ WeighParams p)
{
    using C = Prompt<D>;
    constexpr int NQ = C::NQ;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sb = raw + pad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sQ = sb + C::OFF_Q, bar0 = sb + C::OFF_BAR;
    const uint32_t barK = bar0, barKfree = bar0 + 8;
    auto q_full = [&](int u) { return bar0 + 8u * (2 + u % C::QS); };
    auto q_empty = [&](int u) { return bar0 + 8u * (2 + C::QS + u % C::QS); };
    const uint32_t barS0 = bar0 + 8u * (2 + 2 * C::QS);
    auto s_full = [&](uint32_t t) { return barS0 + 8u * (t % C::NBUF); };
    auto s_free = [&](uint32_t t) { return barS0 + 8u * (C::NBUF + t % C::NBUF); };
    const uint32_t barR0 = barS0 + 16u * C::NBUF;
    auto r_full = [&](uint32_t s) { return barR0 + 8u * (s % C::NR); };
    auto r_free = [&](uint32_t s) { return barR0 + 8u * (C::NR + s % C::NR); };
    const uint32_t barUnit = barR0 + 16u * C::NR, barDone = barUnit + 8;
    float *rows_lse = reinterpret_cast<float *>(smem + C::OFF_ROWS);
    volatile Misc *misc = reinterpret_cast<volatile Misc *>(smem + C::OFF_MISC);
    volatile int *abort_flag = &misc->abort;
    unsigned int *status = &g_weigh_status;
    const uint64_t tmo = p.timeout_ns;

    grid_done_soon();
    if (threadIdx.x == 0) {
        mbar_init(barK, 1);
        mbar_init(barKfree, 1);
        for (int s = 0; s < C::QS; ++s) {
            mbar_init(q_full(s), 1);
            mbar_init(q_empty(s), 1);
        }
        for (int i = 0; i < C::NBUF; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(s_free(i), 4);
        }
        for (int i = 0; i < C::NR; ++i) {
            mbar_init(r_full(i), 1);
            mbar_init(r_free(i), 8);
        }
        mbar_init(barUnit, 1);
        mbar_init(barDone, 1);
        misc->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(const_cast<uint32_t *>(&misc->tmem)), 512);
        tmem_relinquish();
    }
    int total = 0, ctas = 1;   // (warp 3) all steps, the CTAs that share them
    if (warp == 3) {
        grid_wait();
        const Share w = find_share(p.s.B, lane, blockIdx.x, gridDim.x, [&](int b) {
            const WeighLen l = weigh_len(p.s, b);
            return p.s.Hkv * weigh_before(l, l.kt);
        });
        const WeighWalk mine(p.s, w.b, w.off, w.left);
        total = w.total;
        ctas = w.G;
        if (lane == 0) const_cast<Misc *>(misc)->share = mine;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_wait();   // every thread: what it reads and writes from here on may be the kernel's before
    const uint32_t tmem = misc->tmem;
    WeighWalk walk = const_cast<const Misc *>(misc)->share;
    WeighSeg g;

    const WarpWait wait_all{abort_flag, tmo, status};

    if (warp == 0) {
        // ------------------------------------------------------------ K producer, Q producer
        const int boxes = div2(256, p.box_rows);
        const bool inject = (p.inject & 1u) || ((p.inject & 2u) && blockIdx.x == 0);   // the first key tile is left out
        int unit = 0, qu = 0;
        bool ok = true;
        for (; ok && walk.next(p.s, g); ++unit) {
            if (unit) ok = wait_all(barKfree, (unit - 1) & 1, S_KEMPTY);
            if (!ok) break;
            const int valid = inject && unit == 0 ? 0 : min(boxes, cdiv2(g.len.n - g.kt * 256, p.box_rows));
            if (lane == 0 && valid > 0) mbar_arrive_expect_tx(barK, (uint32_t)(valid * p.box_rows * 128 * C::PANELS));
            __syncwarp();
            int pid = 0, row = 0;
            if (lane < valid) page_of(p.pages, g.b, g.kt * 256 + lane * p.box_rows, pid, row);
            load_boxes<C::PANELS>(sb, C::KPANEL, p.box_rows * 128, &maps.k, g.kvh, real_page(p.pages, pid), row, 0, valid, barK);
            WeighTiles t(g);
            for (int s = g.s0; s < g.s1; ++s, t.next(), ++qu) {
                ok = wait_all(q_empty(qu), ((qu / C::QS) & 1) ^ 1, S_QEMPTY);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full(qu), C::QTILE);
#pragma unroll
                    for (int pq = 0; pq < C::PANELS; ++pq)
                        tma_load_3d(sQ + (uint32_t)(qu % C::QS) * C::QTILE + pq * C::QPANEL, &maps.q, pq * 64, t.qt * NQ,
                                    (g.b * p.s.Hkv + g.kvh) * g.len.planes + t.plane, q_full(qu));
                }
            }
        }
        if (lane == 0) {
            if (unit && !(inject && unit == 1)) bounded_wait(barK, (unit - 1) & 1, abort_flag, tmo, S_DRAIN, status, false);
            for (int x = max(0, qu - C::QS); x < qu; ++x) bounded_wait(q_full(x), (x / C::QS) & 1, abort_flag, tmo, S_DRAIN, status, false);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (whole warp)
        constexpr uint32_t HI = sdesc_hi_sw128(1024), id = idesc_f16(BF16, 128, NQ, false);
        int unit = 0, qu = 0;
        uint32_t t = 0;         // score tile
        bool ok = true;
        for (; ok && walk.next(p.s, g); ++unit) {
            ok = wait_all(barK, unit & 1, S_KFULL);
            // the products of the unit before, which read K from tensor memory, are done
            if (ok && unit) ok = wait_all(barUnit, (unit - 1) & 1, S_KEMPTY);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int pn = 0; pn < C::PANELS; ++pn)
                    copy_panel_elect(tmem + h * (D / 2) + pn * 32, sdesc_lo(sb + pn * C::KPANEL + h * 16384, 16), HI);
            tc_commit_elect(barKfree);
            for (int s = g.s0; s < g.s1; ++s, ++qu) {
                ok = wait_all(q_full(qu), (qu / C::QS) & 1, S_QFULL);
                if (!ok) break;
                const uint32_t sq = sQ + (uint32_t)(qu % C::QS) * C::QTILE;
#pragma unroll
                for (int h = 0; h < 2; ++h, ++t) {
                    ok = wait_all(s_free(t), ((t / C::NBUF) & 1) ^ 1, S_FREE);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int pn = 0; pn < C::PANELS; ++pn)
                        mma_ts_k4_elect(tmem + C::COL_S + (t % C::NBUF) * NQ, tmem + h * (D / 2) + pn * 32, sdesc_lo(sq + pn * C::QPANEL, 16),
                                        HI, id, pn ? 1u : 0u);
                    tc_commit_elect(s_full(t));
                }
                if (!ok) break;
                tc_commit_elect(q_empty(qu));
            }
            tc_commit_elect(barUnit);
        }
        tc_commit_elect(barDone);
        bounded_wait(barDone, 0, abort_flag, tmo, S_DRAIN, status, false);
        __syncwarp();
    } else if (warp < 4) {
        // ------------------------------------------------------------ rows: lse and limits, alternate steps
        uint32_t st = 0;
        bool ok = true;
        while (ok && walk.next(p.s, g)) {
            const size_t head0 = (size_t)(g.b * p.s.Hkv + g.kvh) * p.s.group;
            WeighTiles t(g);
            for (int s = g.s0; s < g.s1; ++s, ++st, t.next()) {
                if ((int)(st & 1) != warp - 2) continue;
                float neg[4];
                int limit[4], low = 0x7fffffff;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = 4 * lane + e, i = t.qt * NQ + c;
                    neg[e] = 0.f;
                    limit[e] = 0;
                    if (c < NQ && i < g.len.a) {
                        const float v = p.lse[(head0 + t.plane) * p.s.T + i];
                        neg[e] = v * -1.4426950408889634f;
                        // a row that saw nothing gave nothing
                        limit[e] = v == -INFINITY ? 0 : (p.s.causal ? clampi(g.len.off + i + 1, 0, g.len.n) : g.len.n);
                    }
                    if (c < NQ) low = min(low, limit[e]);
                }
                low = __reduce_min_sync(~0u, low);
                const uint32_t ri = st % C::NR;
                ok = wait_all(r_free(st), ((st / C::NR) & 1) ^ 1, S_FREE);
                if (!ok) break;
                reinterpret_cast<float4 *>(rows_lse + ri * 256)[lane] = make_float4(neg[0], neg[1], neg[2], neg[3]);
                reinterpret_cast<int4 *>(rows_lse + ri * 256 + 128)[lane] = make_int4(limit[0], limit[1], limit[2], limit[3]);
                if (lane == 0) misc->lowest[ri] = low;
                __syncwarp();
                if (lane == 0) mbar_arrive(r_full(st));
            }
        }
        if (warp == 3 && lane == 0) {   // for the joining kernel
            const WeighWalk own = const_cast<const Misc *>(misc)->share;
            Cut c = {};
            if (own.left > 0) c = Cut{own.b, own.kvh, own.kt, parts_from(total, ctas, blockIdx.x, own.s, weigh_steps(own.len, own.kt)), own.len.n, {}};
            p.cuts[blockIdx.x] = c;
        }
    } else {
        // ------------------------------------------------------------ sums, one thread per key
        const int grp = (warp - 4) >> 2, r = (threadIdx.x - 128) & 127;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint64_t sl2x2 = f2_pack(p.sl2, p.sl2);
        uint32_t st = 0;
        bool ok = true;
        while (ok && walk.next(p.s, g)) {
            const int key0 = g.kt * 256 + grp * 128, slot = key0 + r;
            const size_t at = (size_t)(g.b * p.s.Hkv + g.kvh) * p.s.capacity + slot;
            const bool whole = g.s0 == 0 && g.s1 == g.ns, live = slot < g.len.n;
            float base = 0.f, sum = 0.f;
            if (whole && live && p.weight) base = p.weight[at];
            for (int s = g.s0; s < g.s1; ++s, ++st) {
                const uint32_t t = 2 * st + grp, ri = st % C::NR;
                ok = wait_all(r_full(st), (st / C::NR) & 1, S_ROWS) && wait_all(s_full(t), (t / C::NBUF) & 1, S_S);
                if (!ok) break;
                tc_fence_after();
                const float *neg = rows_lse + ri * 256;
                const int *limit = reinterpret_cast<const int *>(neg) + 128;
                const uint32_t tS = tmem + lane_off + C::COL_S + (t % C::NBUF) * NQ;
                uint64_t sum2[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) sum2[i] = f2_pack(0.f, 0.f);
                // 32 columns: exp2(s sl2 - lse2), two columns to an instruction but for the exponential
                auto add = [&](const uint32_t(&sv)[32], int c, bool masked) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const ulonglong2 l = *reinterpret_cast<const ulonglong2 *>(neg + c + e);
                        float x[4];
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), sl2x2, l.x), x[0], x[1]);
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[e + 2]), __uint_as_float(sv[e + 3])), sl2x2, l.y), x[2], x[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[i] = ex2_approx(x[i]);
                        if (masked) {
                            const int4 m = *reinterpret_cast<const int4 *>(limit + c + e);
                            x[0] = slot < m.x ? x[0] : 0.f;
                            x[1] = slot < m.y ? x[1] : 0.f;
                            x[2] = slot < m.z ? x[2] : 0.f;
                            x[3] = slot < m.w ? x[3] : 0.f;
                        }
                        sum2[(e >> 1) & 3] = f2_add(sum2[(e >> 1) & 3], f2_pack(x[0], x[1]));
                        sum2[((e >> 1) + 1) & 3] = f2_add(sum2[((e >> 1) + 1) & 3], f2_pack(x[2], x[3]));
                    }
                };
                if (misc->lowest[ri] >= key0 + 128) {
                    // every row sees the whole key tile: the next 32 columns are read while these are summed
                    uint32_t va[32], vb[32];
                    tmem_ld_x32(tS, va);
                    tmem_wait_ld();
                    reg_fence_x32(va);
#pragma unroll(LONG ? NQ / 64 : 1)
                    for (int c = 0; c < NQ; c += 64) {
                        tmem_ld_x32(tS + c + 32, vb);
                        add(va, c, false);
                        tmem_wait_ld();
                        reg_fence_x32(vb);
                        if (c + 64 < NQ) tmem_ld_x32(tS + c + 64, va);
                        add(vb, c + 32, false);
                        if (c + 64 < NQ) {
                            tmem_wait_ld();
                            reg_fence_x32(va);
                        }
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < NQ; c += 32) {
                        uint32_t sv[32];
                        tmem_ld_x32(tS + c, sv);
                        tmem_wait_ld();
                        reg_fence_x32(sv);
                        add(sv, c, true);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(s_free(t));
                    mbar_arrive(r_free(st));
                }
                float la, lb;
                f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), la, lb);
                sum += la + lb;
            }
            if (!ok) break;
            if (live) {
                if (whole)
                    p.out[at] = base + sum;
                else
                    p.part[(size_t)part_slot(blockIdx.x, g.s0) * 256 + grp * 128 + r] = sum;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    } else if (warp >= 4 && *abort_flag) {
        // This CTA gave up on a wait: NaN into every sum it was given
        const int r = threadIdx.x - 128;
        walk = const_cast<const Misc *>(misc)->share;
        while (walk.next(p.s, g)) {
            const int slot = g.kt * 256 + r;
            if (slot >= g.len.n) continue;
            if (g.s0 == 0 && g.s1 == g.ns)
                p.out[(size_t)(g.b * p.s.Hkv + g.kvh) * p.s.capacity + slot] = __uint_as_float(~0u);
            else
                p.part[(size_t)part_slot(blockIdx.x, g.s0) * 256 + r] = __uint_as_float(~0u);
        }
    }
}

// Adds the parts of the key tiles that a cut crosses, in the order of the steps; block x looks whether CTA
// x + 1 left such a key tile (its first cut is the start of that CTA's share).
__global__ void __launch_bounds__(256) weigh_join_kernel(const __grid_constant__ WeighParams p)
{
    const int r = threadIdx.x;
    grid_wait();
    grid_done_soon();
    const Cut c = p.cuts[blockIdx.x + 1];
    const int slot = c.tile * p.s.keys + r;
    if (c.parts == 0 || slot >= c.n) return;
    const size_t at = (size_t)(c.b * p.s.Hkv + c.kvh) * p.s.capacity + slot;
    const float base = p.weight ? p.weight[at] : 0.f;
    float sum = 0.f;
#pragma unroll 4
    for (int i = 0; i < c.parts; ++i) sum += p.part[(size_t)part_slot((int)blockIdx.x + i, i) * 256 + r];
    p.out[at] = base + sum;
}

// KIND 0: gathered or packed rows; 1: a prompt; 2: a long prompt, with the loop over a tile's columns
// unrolled: 208 instead of 228 us for 8192 tokens (32 heads, D = 128), but 33 instead of 29 us for
// 2048 and 26 instead of 20 us for 8 x 300, where fetching the longer code is what counts.
constexpr int kLongPrompt = 4096;

template <int D, bool BF16, int KIND>
cudaError_t launch_one(const WeighMaps &m, const WeighParams &p0, cudaStream_t st)
{
    auto kern = KIND == 0 ? weigh_kernel<D, BF16> : weigh_prompt_kernel<D, BF16, KIND == 2>;
    constexpr int threads = KIND ? Prompt<D>::THREADS : THREADS, smem = KIND ? Prompt<D>::ALLOC : Cfg<D>::ALLOC;
    static std::atomic<uint64_t> configured{0};
    static std::atomic<int> sm_count[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const uint64_t bit = 1ull << dev;
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        int nsm = 0;
        e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        sm_count[dev].store(nsm, std::memory_order_relaxed);
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    WeighParams p = p0;
    if (p.timeout_ns == 0) p.timeout_ns = kDefaultTimeoutNs;
    const int grid = clampi(sm_count[dev].load(std::memory_order_relaxed), 1, kMaxCtas);
    e = launch_overlapped(kern, dim3(grid), threads, smem, 1, st, m, p);
    if (e != cudaSuccess || grid == 1) return e;
    return launch_overlapped(weigh_join_kernel, dim3(grid - 1), p.s.keys, 0, 1, st, p);
}

} // namespace

int weigh_rows(int D) { return D == 256 ? 64 : 128; }

cudaError_t launch_weigh(int D, bool bf16, const WeighMaps &m, const WeighParams &p, cudaStream_t st)
{
    const int kind = p.s.mode != kHeads ? 0 : (p.s.T >= kLongPrompt && D != 256 ? 2 : 1);   // D = 256: one iteration either way
#define WEIGH_CASE(DD, BB, KK) \
    if (D == DD && bf16 == BB && kind == KK) return launch_one<DD, BB, KK>(m, p, st);
    WEIGH_CASE(64, true, 0) WEIGH_CASE(64, true, 1) WEIGH_CASE(64, true, 2)
    WEIGH_CASE(64, false, 0) WEIGH_CASE(64, false, 1) WEIGH_CASE(64, false, 2)
    WEIGH_CASE(128, true, 0) WEIGH_CASE(128, true, 1) WEIGH_CASE(128, true, 2)
    WEIGH_CASE(128, false, 0) WEIGH_CASE(128, false, 1) WEIGH_CASE(128, false, 2)
    WEIGH_CASE(256, true, 0) WEIGH_CASE(256, true, 1) WEIGH_CASE(256, false, 0) WEIGH_CASE(256, false, 1)
#undef WEIGH_CASE
    return cudaErrorInvalidValue;
}

cudaError_t read_and_clear_weigh_status(uint32_t *word)
{
    unsigned int w = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&w, g_weigh_status, sizeof(w));
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_weigh_status, &zero, sizeof(zero));
    if (word) *word = w;
    return e;
}

} // namespace cache
} // namespace fa
