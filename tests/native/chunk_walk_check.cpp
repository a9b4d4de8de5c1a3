// Host check of what shares do with their cuts (chunk_schedule.h): every key tile of every item is
// walked once, whole items are whole, and of an item that is cut the joining reads just the states
// that its pieces leave, in the order of the keys, each from a place of its own.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <set>
#include <utility>
#include <vector>

#include "chunk_schedule.h"

using namespace pkv::chunk;

namespace {

int fail(const char *what, long a, long b)
{
    std::printf("%s: %ld %ld\n", what, a, b);
    return 1;
}

struct Item {
    int b, h, rt, lo, hi, tok, rows;
    int64_t at;
};

// A share's state of an item: which of its two, and the tiles that are in it.
struct State {
    int share, slot, t0, t1;
};

int check_batch(unsigned seed)
{
    std::srand(seed);
    Rules r;
    const int lg_g = std::rand() % 4;
    r.lg_tpr = (std::rand() % 2 ? 8 : 7) - lg_g;
    r.tree = std::rand() % 4 == 0;
    r.window = !r.tree && std::rand() % 2 ? 1 + std::rand() % (std::rand() % 4 ? 700 : 1 << 30) : 0;
    const int B = 1 + std::rand() % 7, H = 1 + std::rand() % 3, most = seed % 5 == 0 ? 40000 : 3000;
    std::vector<Seq> seqs(B);
    std::vector<int> q0(B);
    int tokens = std::rand() % 4;
    for (int b = 0; b < B; ++b) {
        Seq &q = seqs[b];
        q.n = r.tree ? std::rand() % 65 : std::rand() % 4 == 0 ? 0 : std::rand() % 3 ? std::rand() % 9 : std::rand() % 2000;
        q.L = q.n + (std::rand() % 3 ? std::rand() % most : 0);
        q0[b] = tokens;
        tokens += q.n;
    }
    auto lengths = [&](int b, Seq &q, int &at) {
        q = seqs[b];
        at = q0[b];
        return q.n > 0;
    };
    std::vector<Item> items;
    std::vector<int64_t> start(B + 1);
    int64_t U = 0;
    for (int b = 0; b < B; ++b) {
        start[b] = U;
        for (int h = 0; h < H && seqs[b].n > 0; ++h)
            for (int rt = 0; rt < row_tiles(r, seqs[b]); ++rt) {
                const int tpr = 1 << r.lg_tpr, left = seqs[b].n - rt * tpr;
                Item i{b, h, rt, 0, 0, q0[b] + rt * tpr, (left < tpr ? left : tpr) << lg_g, U};
                tiles(r, seqs[b], rt, i.lo, i.hi);
                items.push_back(i);
                U += i.hi - i.lo + ITEM_COST;
            }
    }
    start[B] = U;
    if (U == 0)
        return 0;
    const int ctas = 1 + std::rand() % 200, n = shares(U, ctas);
    const uint32_t step = share_step(ctas);
    // the place of a share's start, as the kernel finds it
    auto place = [&](int c) {
        const int64_t x = share_start(U, n, c, ctas, step);
        Place p{};
        p.b = B;
        for (int b = 0; b < B && c < n; ++b)
            if (x >= start[b] && x < start[b + 1])
                p = place_in(r, seqs[b], b, x - start[b], cost_of(r, seqs[b]));
        return p;
    };
    for (int c = 0; c < n; ++c)
        if (n > 1 && share_start(U, n, c + 1, ctas, step) - share_start(U, n, c, ctas, step) < MIN_SHARE)
            return fail("share", c, n);
    // all shares' walks
    std::map<std::vector<int>, std::vector<State>> states;
    std::map<std::vector<int>, std::vector<int>> seen;         // of an item: how often each tile was
    for (const Item &i : items)
        seen[{i.b, i.h, i.rt}] = std::vector<int>(i.hi - i.lo);
    for (int c = 0; c < n; ++c) {
        const Place places[2] = {place(c), place(c + 1)};
        Walk walk{};
        walk.start(B, places, lengths);
        std::set<int> slots;
        Piece p;
        for (int k = 0; walk.next(r, B, H, lg_g, p, lengths); ++k) {
            const int rt = (p.tok - q0[p.b]) >> r.lg_tpr;
            const std::vector<int> key = {p.b, p.h, rt};
            if (!seen.count(key))
                return fail("no such item", p.b, p.tok);
            std::vector<int> &of = seen[key];
            int lo, hi, first, last;
            tiles(r, seqs[p.b], rt, lo, hi);
            span(r, seqs[p.b], rt, first, last);
            if (p.t0 < lo || p.t1 > hi || p.t0 >= p.t1)
                return fail("tiles", p.t0, p.t1);
            if (p.first != first || p.last != last || p.len != seqs[p.b].L || p.base != p.len - seqs[p.b].n ||
                p.sight != (r.window > 0 && first >= r.window ? first - r.window + 1 : 0))
                return fail("piece", p.b, p.tok);
            const int tpr = 1 << r.lg_tpr, left = seqs[p.b].n - rt * tpr;
            if (p.tok != q0[p.b] + rt * tpr || p.rows != (left < tpr ? left : tpr) << lg_g)
                return fail("rows", p.tok, p.rows);
            for (int t = p.t0; t < p.t1; ++t)
                ++of[t - lo];
            const bool whole = p.t0 == lo && p.t1 == hi;
            if ((p.kind == 0) != whole || (p.kind == 1) != (p.t0 > lo))
                return fail("kind", p.kind, p.t0 - lo);
            if (whole)
                continue;
            // the first of its pieces, or its last: one state each
            const int slot = p.kind == 2;
            if (!slots.insert(slot).second || (slot == 0 && k > 0))
                return fail("slot", c, slot);
            states[key].push_back({c, slot, p.t0, p.t1});
        }
    }
    for (const auto &s : seen)
        for (int x : s.second)
            if (x != 1)
                return fail("a tile's times", x, s.first[2]);
    // what the joining reads
    size_t joined = 0;
    for (int c = 0; c < n; ++c) {
        const Place a = place(c);
        if (!a.split)
            continue;
        const int pieces = pieces_to_join(r, seqs[a.b], a, U, n, c, ctas, step);
        if (pieces == 0)
            continue;
        ++joined;
        const std::vector<State> &of = states[{a.b, a.h, a.rt}];
        if ((int)of.size() != pieces)
            return fail("pieces", pieces, (long)of.size());
        int t = 0, hi;
        tiles(r, seqs[a.b], a.rt, t, hi);
        for (int i = 0; i < pieces; ++i) {
            if (of[i].share != c - 1 + i || of[i].slot != (i == 0) || of[i].t0 != t)
                return fail("state", c, i);
            t = of[i].t1;
        }
        if (t != hi)
            return fail("keys", t, hi);
    }
    if (joined != states.size())
        return fail("items joined", (long)joined, (long)states.size());
    return 0;
}

}  // namespace

int main()
{
    for (unsigned seed = 1; seed <= 4000; ++seed)
        if (check_batch(seed)) {
            std::printf("seed %u\n", seed);
            return 1;
        }
    std::printf("ok\n");
    return 0;
}
