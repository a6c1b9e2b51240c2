// Host-side check of csrc/cache_schedule.h, built and run by tests/test_cache_cpu.py: under random
// shapes, every step of every unit is given to exactly one CTA, CTAs get equal shares, the parts of a
// cut unit lie in slots that no other part uses, and they are the parts that the joining kernel adds.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <set>
#include <vector>

#include "cache_schedule.h"

using namespace fa::cache;

static int fail(const char *what) { std::printf("FAILED: %s\n", what); return 1; }

static unsigned rnd(unsigned n) { return (unsigned)rand() % n; }

// What find_share of the kernel computes, one sequence at a time.
static TreeWalk share(const TreeShape &s, int least, int grid, int cta, int *total_out, int *G_out)
{
    int total = 0;
    for (int b = 0; b < s.B; ++b) total += s.Hkv * s.units * tree_len(s, b).nt;
    const int G = ctas(total, grid, least);
    int begin = cta < G ? cut(total, G, cta) : total, b = 0;
    const int left = cta < G ? cut(total, G, cta + 1) - begin : 0;
    for (; b < s.B; ++b) {
        const int one = s.Hkv * s.units * tree_len(s, b).nt;
        if (begin < one) break;
        begin -= one;
    }
    *total_out = total;
    *G_out = G;
    return TreeWalk(s, b, begin, left);
}

static int check_tree()
{
    for (int round = 0; round < 400; ++round) {
        std::vector<int32_t> len(1 + rnd(9)), draft(len.size());
        TreeShape s;
        s.B = (int)len.size();
        s.Hkv = 1 + rnd(4);
        s.T = 1 + rnd(200);
        s.rows = s.T * (1 + rnd(4));
        s.tile = rnd(2) ? 128 : 256;
        s.units = cdiv(s.rows, s.tile);
        s.lbn = rnd(2) ? 7 : 6;
        s.capacity = 16 * (1 + rnd(300));
        for (size_t b = 0; b < len.size(); ++b) {
            len[b] = (int)rnd(s.capacity + 40) - 20;   // out of range on both sides, too
            draft[b] = (int)rnd(s.T + 4) - 2;
        }
        s.seq_len = len.data();
        s.draft_len = rnd(4) ? draft.data() : nullptr;
        const int grid = 1 + rnd(160), least = 1 + rnd(4);
        std::map<long long, std::vector<int>> unit;          // (b, kvh, mt) -> owner of each step
        std::map<long long, std::vector<std::pair<int, int>>> parts;   // -> (k0, slot) of its parts
        std::set<int> used;
        int total = 0, G = 0, given = 0, most = 0, fewest = 1 << 30;
        for (int c = 0; c < grid; ++c) {
            TreeWalk w = share(s, least, grid, c, &total, &G);
            int mine = 0;
            TreeSeg g;
            while (w.next(s, g)) {
                const long long id = ((long long)g.b * s.Hkv + g.kvh) * s.units + g.mt;
                if (g.len.nt <= 0 || g.k0 < 0 || g.k1 <= g.k0 || g.k1 > g.len.nt || g.kvh >= s.Hkv || g.mt >= s.units)
                    return fail("a segment outside its unit");
                auto &own = unit[id];
                own.resize(g.len.nt, -1);
                for (int k = g.k0; k < g.k1; ++k) {
                    if (own[k] != -1) return fail("a step given twice");
                    own[k] = c;
                }
                if (!(g.k0 == 0 && g.k1 == g.len.nt)) {
                    const int slot = part_slot(c, g.k0);
                    if (!used.insert(slot).second || slot >= 2 * grid) return fail("a part's slot");
                    parts[id].push_back({g.k0, slot});
                }
                mine += g.k1 - g.k0;
            }
            if (c < G) {
                most = mine > most ? mine : most;
                fewest = mine < fewest ? mine : fewest;
            } else if (mine) {
                return fail("work behind the last CTA");
            }
            given += mine;
        }
        if (given != total) return fail("steps that nobody has");
        if (total && most - fewest > 1) return fail("unequal shares");
        size_t units = 0;
        for (int b = 0; b < s.B; ++b) units += tree_len(s, b).nt ? (size_t)s.Hkv * s.units : 0;
        if (unit.size() != units) return fail("units that nobody has");
        for (auto &u : unit)
            for (int o : u.second)
                if (o < 0) return fail("a step that nobody has");
        // the joining kernel's view: block k of cut k
        size_t joined = 0;
        for (int k = 1; k < grid; ++k) {
            int t2, G2;
            TreeWalk w = share(s, least, grid, k, &t2, &G2);
            TreeSeg g;
            if (k >= G2 || !w.next(s, g)) continue;
            const int n = parts_from(t2, G2, k, g.k0, g.len.nt);
            if (n == 0) continue;
            const auto &want = parts[((long long)g.b * s.Hkv + g.kvh) * s.units + g.mt];
            if ((int)want.size() != n) return fail("the number of parts");
            for (int i = 0; i < n; ++i)
                if (part_slot(k - 1 + i, i) != want[i].second) return fail("the order of the parts");
            ++joined;
        }
        if (joined != parts.size()) return fail("a cut unit that is not joined");
        for (int step = 0; step < total; step += 1 + rnd(50)) {
            const int c = cta_of(total, G, step);
            if (cut(total, G, c) > step || cut(total, G, c + 1) <= step) return fail("the CTA of a step");
        }
    }
    return 0;
}

static int check_weigh()
{
    for (int round = 0; round < 400; ++round) {
        std::vector<int32_t> len(1 + rnd(6)), count(len.size());
        WeighShape s;
        s.B = (int)len.size();
        s.Hkv = 1 + rnd(3);
        s.group = 1 + rnd(4);
        s.T = 1 + rnd(rnd(2) ? 20 : 700);
        s.mode = rnd(3);
        s.causal = rnd(3) != 0;
        s.NQ = rnd(2) ? 128 : 64;
        s.keys = s.mode == kHeads ? 256 : 128;
        s.capacity = 16 * (1 + rnd(60));
        for (size_t b = 0; b < len.size(); ++b) {
            len[b] = (int)rnd(s.capacity + 20) - 10;
            count[b] = (int)rnd(s.T + 4) - 2;
        }
        s.seq_len = len.data();
        s.count = rnd(4) ? count.data() : nullptr;
        std::vector<int> base;
        int total = 0;
        for (int b = 0; b < s.B; ++b) {
            const WeighLen l = weigh_len(s, b);
            base.push_back(total);
            int sum = 0;
            for (int k = 0; k < l.kt; ++k) {
                if (weigh_before(l, k) != sum) return fail("the steps before a key tile");
                if (weigh_steps(l, k) < 1) return fail("a key tile without steps");
                sum += weigh_steps(l, k);
            }
            if (weigh_before(l, l.kt) != sum) return fail("the steps of a head");
            total += s.Hkv * sum;
        }
        const int grid = 1 + rnd(160), least = 1 + rnd(3), G = ctas(total, grid, least);
        std::map<long long, std::set<int>> seen;   // (b, kvh, kt) -> its steps
        std::map<long long, std::set<std::pair<int, int>>> tiles;
        for (int c = 0; c < G; ++c) {
            const int begin = cut(total, G, c);
            int b = 0;
            while (b + 1 < s.B && base[b + 1] <= begin) ++b;
            WeighWalk w(s, b, begin - base[b], cut(total, G, c + 1) - begin);
            WeighSeg g;
            while (w.next(s, g)) {
                const long long id = ((long long)g.b * s.Hkv + g.kvh) * 100000 + g.kt;
                if (g.s0 < 0 || g.s1 <= g.s0 || g.s1 > g.ns || g.kt * s.keys >= g.len.n) return fail("a segment outside its unit");
                WeighTiles t(g);
                for (int i = g.s0; i < g.s1; ++i, t.next()) {
                    if (!seen[id].insert(i).second) return fail("a step given twice");
                    const int plane = t.plane, qt = t.qt;
                    if (plane < 0 || plane >= g.len.planes || qt < 0 || (g.len.qt && qt >= g.len.qt)) return fail("a query tile");
                    tiles[id].insert({plane, qt});
                }
            }
            if (s.mode == kHeads) continue;
            // the same share a head at a time
            WeighWalk v(s, b, begin - base[b], cut(total, G, c + 1) - begin), u(s, b, begin - base[b], cut(total, G, c + 1) - begin);
            WeighRun r;
            while (v.next_run(s, r)) {
                if (r.steps < 1 || r.len.planes != 1) return fail("a run");
                for (int i = 0, kt = r.kt, at = r.s; i < r.steps;) {
                    if (!u.next(s, g) || g.b != r.b || g.kvh != r.kvh || g.kt != kt || g.s0 != at || g.ns != r.ns || g.first != 0)
                        return fail("a run and its segments");
                    i += g.s1 - g.s0;
                    at = 0;
                    ++kt;
                    if (i > r.steps) return fail("a run's end");
                }
            }
            if (u.next(s, g)) return fail("a segment without a run");
        }
        // every row that sees a slot of a key tile lies in one of the unit's query tiles
        for (int b = 0; b < s.B; ++b) {
            const WeighLen l = weigh_len(s, b);
            for (int h = 0; h < s.Hkv; ++h)
                for (int k = 0; k < l.kt; ++k) {
                    const long long id = ((long long)b * s.Hkv + h) * 100000 + k;
                    if ((int)seen[id].size() != weigh_steps(l, k)) return fail("a step that nobody has");
                    for (int plane = 0; plane < l.planes; ++plane)
                        for (int r = 0; r < l.rows; ++r) {
                            const bool sees = s.mode != kHeads || !s.causal || s.keys * k < l.off + r + 1;
                            if (sees && !tiles[id].count({plane, r / s.NQ})) return fail("a row that is left out");
                        }
                }
        }
    }
    return 0;
}

static int check_cuts()
{
    // both widths of the arithmetic, and the line between them
    for (int total : {1, 2, 159, 8388607, 8388608, 8388609, 2147483647})
        for (int G : {1, 2, 151, 152, 160})
            for (int c = 0; c <= G && total >= G; ++c) {
                if (cut(total, G, c) != (int)((long long)total * c / G)) return fail("a cut");
                if (c < G && (cta_of(total, G, cut(total, G, c)) != c || (c && cta_of(total, G, cut(total, G, c) - 1) != c - 1))) return fail("the CTA of a cut");
            }
    return 0;
}

int main()
{
    srand(1);
    if (check_cuts() || check_tree() || check_weigh()) return 1;
    std::printf("ok\n");
    return 0;
}
