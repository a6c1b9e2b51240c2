// bwd_schedule_check.cpp -- host-side check of the backward pass's work schedule (bwd_internal.h), built and run by
// tests/test_bwd_cpu.py.
//
// For each shape, mask and grid it walks every CTA's rounds as the kernels do and checks that every part of every (plane,
// tile) is visited once, that a unit's parts read each streamed tile that holds an allowed pair exactly once, of the right
// planes, in order, and tiles without one not at all (but for a ragged last tile's padding rows), and that parts fit the workspace.
#include <cstdio>
#include <map>
#include <set>
#include <vector>

#include "bwd_internal.h"

using namespace fa::bwd;

static int fails = 0;
#define CHECK(x) do { if (!(x) && fails++ < 20) std::printf("FAIL %s: B=%d Hq=%d Hkv=%d Sq=%d Sk=%d D=%d causal=%d rowq=%d G=%d\n", #x, B, Hq, Hkv, Sq, Sk, D, causal, (int)rowq, G); } while (0)

template <bool rowq, int BN>
static void walk(int B, int Hq, int Hkv, int Sq, int Sk, int D, int causal, int G)
{
    const Shape s = make_shape(rowq, B, Hq, Hkv, Sq, Sk, D, causal);
    const int group = Hq / Hkv;
    CHECK(s.parts >= 1 && (s.parts == 1 || s.num <= kMaxParts));
    std::vector<int> seen_slots(s.num, 0);
    std::map<std::pair<int, int>, std::vector<std::pair<int, std::vector<std::pair<int, int>>>>> tiles;
    for (int c = 0; c < G; ++c) {
        Unit u;
        for (int round = 0; unit_at<rowq, BN>(s, G, c, round, u); ++round) {
            CHECK(u.z >= 0 && u.z < s.planes && u.t >= 0 && u.t < s.tiles && u.slot >= 0 && u.slot < s.num && u.n >= 0);
            if (u.slot < 0 || u.slot >= s.num) continue;
            seen_slots[u.slot]++;
            std::vector<std::pair<int, int>> at;
            int plane = u.plane, tile = u.tile;
            for (int j = 0; j < u.n; ++j) {
                at.push_back({plane, tile});
                if (++tile == u.end) {
                    tile = u.first;
                    ++plane;
                }
            }
            tiles[{u.z, u.t}].push_back({u.slot % s.parts, at});
        }
    }
    for (int x : seen_slots) CHECK(x == 1);
    const long long off = causal == 2 ? Sk - Sq : 0;
    for (auto &it : tiles) {
        const int z = it.first.first, t = it.first.second;
        std::map<int, std::vector<std::pair<int, int>>> by;
        for (auto &p : it.second) by[p.first] = p.second;
        std::vector<std::pair<int, int>> got;
        for (auto &p : by) got.insert(got.end(), p.second.begin(), p.second.end());
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
                        }
    std::printf(fails ? "%d failures\n" : "ok\n", fails);
    return fails != 0;
}
