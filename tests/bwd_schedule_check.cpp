// bwd_schedule_check.cpp -- host-side check of the backward pass's work schedule (bwd_internal.h), built and run by
// tests/test_bwd_cpu.py.
//
// For each shape, mask and grid it walks every CTA's rounds as the kernels do and checks that every (plane, tile), or every
// part of it, is visited once, that a unit's parts read each streamed tile that holds an allowed pair exactly once, of the right
// planes, in order, and tiles without one not at all (but for a ragged last tile's padding rows), and that the parts
// that are joined are those that are left.
#include <cstdio>
#include <map>
#include <set>
#include <vector>

#include "bwd_internal.h"

using namespace fa::bwd;

static int fails = 0;
#define CHECK(x) do { if (!(x) && fails++ < 20) std::printf("FAIL %s: B=%d Hq=%d Hkv=%d Sq=%d Sk=%d D=%d causal=%d rowq=%d G=%d\n", #x, B, Hq, Hkv, Sq, Sk, D, causal, (int)rowq, G); } while (0)

template <bool rowq, int BN>
static void walk(int B, int Hq, int Hkv, int Sq, int Sk, int D, int causal, int G, bool cut = false)
{
    const Shape s = make_shape(rowq, B, Hq, Hkv, Sq, Sk, D, causal);
    const int group = Hq / Hkv;
    Cuts cuts = {};
    Join join = {};
    if (cut) {
        const Load l = load_of<rowq, BN>(s);
        if (l.total == 0) return;
        cut_evenly<rowq, BN>(s, l, cuts, join);
        G = cuts.ctas;
    }
    const int slots = parts_of(cuts);
    CHECK(G <= kCtas && slots <= 2 * kCtas && join.num <= kCtas && (!cut || join.slot[join.num] == slots));
    std::vector<int> seen_slots(slots, 0);
    // the parts of each unit, in the order of their slots
    std::map<std::pair<int, int>, std::map<int, std::vector<std::pair<int, int>>>> tiles;
    std::map<std::pair<int, int>, int> number;
    std::vector<int> load(G, 0);
    for (int c = 0; c < G; ++c) {
        Unit u;
        for (int round = 0; unit_at<rowq, BN>(s, cuts, G, c, round, u); ++round) {
            CHECK(u.z >= 0 && u.z < s.planes && u.t >= 0 && u.t < s.tiles && u.slot >= -1 && u.slot < slots && u.n >= 0);
            if (u.slot >= 0 && u.slot < slots) seen_slots[u.slot]++;
            std::vector<std::pair<int, int>> at;
            int plane = u.plane, tile = u.tile;
            for (int j = 0; j < u.n; ++j) {
                at.push_back({plane, tile});
                if (++tile == u.end) {
                    tile = u.first;
                    ++plane;
                }
            }
            auto &of = tiles[{u.z, u.t}];
            CHECK(of.find(u.slot) == of.end() && (of.empty() || u.slot >= 0));
            of[u.slot] = at;
            load[c] += u.n > 0 ? u.n + kUnitCost : 0;
            CHECK(u.slot < 0 || u.n > 0);
        }
    }
    if (cut)
        for (int x : load) CHECK(x <= load[0] + 2 * kUnitCost + 1);   // shares alike but for what a cut inside a unit repeats
    for (int x : seen_slots) CHECK(x == 1);
    for (int i = 0; i < join.num; ++i) {   // each cut unit's parts, and no others
        const int w = join.unit[i], q = s.causal ? w / s.planes : 0;
        const int t = s.causal ? (rowq ? s.tiles - 1 - q : q) : w % s.tiles, z = s.causal ? w % s.planes : w / s.tiles;
        auto &of = tiles[{z, t}];
        CHECK((int)of.size() == join.slot[i + 1] - join.slot[i] && of.size() > 1 && of.begin()->first == join.slot[i] && of.rbegin()->first == join.slot[i + 1] - 1);
    }
    int cut_units = 0;
    for (auto &it : tiles) cut_units += it.second.begin()->first >= 0;
    CHECK(cut_units == join.num);
    const long long off = causal == 2 ? Sk - Sq : 0;
    for (auto &it : tiles) {
        const int z = it.first.first, t = it.first.second;
        std::vector<std::pair<int, int>> got;
        for (auto &p : it.second) got.insert(got.end(), p.second.begin(), p.second.end());
        std::vector<std::pair<int, int>> want, may;
        const int b = z / s.heads, h = z % s.heads;
        const int p0 = rowq ? b * Hkv + h / group : b * Hq + h * group, np = rowq ? 1 : group;
        for (int p = p0; p < p0 + np; ++p)
            for (int x = 0; x * BN < s.cols; ++x) {
                bool need = false, could = false;
                for (int r = t * kRows; r < t * kRows + kRows && !need; r += 1) {
                    // the streamed rows that row r meets: [lo, hi]
                    long long lo = 0, hi = s.cols - 1;
                    if (causal && rowq && r + off < hi) hi = r + off;
                    if (causal && !rowq && r - off > lo) lo = r - off;
                    const bool meets = lo <= hi && lo < (long long)(x + 1) * BN && hi >= (long long)x * BN;
                    could |= meets;
                    need |= meets && r < s.rows;
                }
                if (need) want.push_back({p, x});
                if (could) may.push_back({p, x});
            }
        CHECK(got == want || got == may);
        for (auto &p : got) CHECK(p.first >= p0 && p.first < p0 + np && p.second >= 0 && p.second * BN < s.cols);
    }
    CHECK((int)tiles.size() == s.planes * s.tiles);
}

int main()
{
    const int lens[] = {1, 2, 63, 64, 65, 127, 128, 129, 200, 256, 300, 513, 700};
    const int heads[][2] = {{1, 1}, {2, 2}, {4, 2}, {6, 1}, {14, 2}};
    for (int B : {1, 3})
        for (auto &h : heads)
            for (int Sq : lens)
                for (int Sk : lens)
                    for (int causal = 0; causal < 3; ++causal)
                        for (int G : {1, 7, 152}) {
                            walk<true, 128>(B, h[0], h[1], Sq, Sk, 128, causal, G);
                            walk<false, 128>(B, h[0], h[1], Sq, Sk, 128, causal, G);
                            walk<true, 64>(B, h[0], h[1], Sq, Sk, 256, causal, G);
                            walk<false, 64>(B, h[0], h[1], Sq, Sk, 256, causal, G);
                            if (G == 1) {
                                walk<true, 128>(B, h[0], h[1], Sq, Sk, 128, causal, 0, true);
                                walk<false, 128>(B, h[0], h[1], Sq, Sk, 128, causal, 0, true);
                                walk<true, 64>(B, h[0], h[1], Sq, Sk, 256, causal, 0, true);
                                walk<false, 64>(B, h[0], h[1], Sq, Sk, 256, causal, 0, true);
                            }
                        }
    // long lines over few units, and units without steps
    const int wide[][6] = {{1, 1, 1, 1, 20000, 0}, {1, 2, 2, 130, 9000, 2}, {1, 8, 1, 2048, 2048, 1}, {2, 14, 2, 1000, 5000, 2}, {1, 1, 1, 9000, 130, 1}, {1, 1, 1, 9000, 130, 2},
                           {3, 6, 2, 700, 1900, 1}, {1, 4, 4, 4096, 4096, 1}, {1, 16, 4, 300, 7000, 0}, {1, 2, 1, 100, 16000, 1}, {5, 32, 8, 1024, 1024, 1}, {1, 3, 1, 5000, 300, 2}};
    for (auto &w : wide)
        for (int causal : {w[5], 0, 1, 2}) {
            walk<true, 128>(w[0], w[1], w[2], w[3], w[4], 128, causal, 0, true);
            walk<false, 128>(w[0], w[1], w[2], w[3], w[4], 128, causal, 0, true);
            walk<true, 64>(w[0], w[1], w[2], w[3], w[4], 256, causal, 0, true);
            walk<false, 64>(w[0], w[1], w[2], w[3], w[4], 256, causal, 0, true);
        }
    std::printf(fails ? "%d failures\n" : "ok\n", fails);
    return fails != 0;
}
