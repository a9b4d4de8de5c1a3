// Host check of chunk_schedule.h: closed forms against sums item by item, and that the shares
// cover every key tile of every item once.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "chunk_schedule.h"

using namespace pkv::chunk;

namespace {

struct Item {
    int b, h, rt, lo, hi;
    int64_t at;
};

int fail(const char *what, long a, long b)
{
    std::printf("%s: %ld %ld\n", what, a, b);
    return 1;
}

int check_batch(unsigned seed)
{
    std::srand(seed);
    Rules r;
    r.lg_tpr = 4 + std::rand() % 5;
    r.tree = std::rand() % 4 == 0;
    r.window = !r.tree && std::rand() % 2 ? 1 + std::rand() % 700 : 0;
    const int B = 1 + std::rand() % 6, H = 1 + std::rand() % 3;
    std::vector<Seq> seqs(B);
    for (Seq &q : seqs) {
        q.n = r.tree ? std::rand() % 65 : std::rand() % 5 == 0 ? 0 : std::rand() % 2000;
        q.L = q.n + (std::rand() % 3 ? std::rand() % 3000 : 0);
    }
    // the line, item by item
    std::vector<Item> items;
    std::vector<int64_t> start(B);
    int64_t U = 0;
    for (int b = 0; b < B; ++b) {
        start[b] = U;
        if (seqs[b].n == 0)
            continue;
        const int64_t one = cost_of(r, seqs[b]);
        for (int h = 0; h < H; ++h)
            for (int rt = 0; rt < row_tiles(r, seqs[b]); ++rt) {
                Item i{b, h, rt, 0, 0, U};
                tiles(r, seqs[b], rt, i.lo, i.hi);
                if (U - start[b] - h * one != cost_before(r, seqs[b], rt))
                    return fail("cost before", U, rt);
                items.push_back(i);
                U += i.hi - i.lo + ITEM_COST;
            }
        if (U - start[b] != H * one)
            return fail("cost", U - start[b], H * one);
    }
    // every position of it
    size_t k = 0;
    for (int64_t x = 0; x < U; ++x) {
        while (k + 1 < items.size() && items[k + 1].at <= x)
            ++k;
        const Item &i = items[k];
        const Place p = place_in(r, seqs[i.b], i.b, x - start[i.b], cost_of(r, seqs[i.b]));
        const int tile = i.lo + (int)(x - i.at > ITEM_COST ? x - i.at - ITEM_COST : 0);
        if (p.b != i.b || p.h != i.h || p.rt != i.rt || p.tile != tile || p.split != (tile > i.lo) ||
            tile >= i.hi)
            return fail("place", x, tile);
    }
    // the cuts: ascending, from 0 to U, none shorter than MIN_SHARE but a line's only one
    const int ctas = 1 + std::rand() % 200, n = shares(U, ctas);
    const uint32_t step = share_step(ctas);
    int64_t before = 0;
    if (U > 0 && share_start(U, n, 0, ctas, step) != 0)
        return fail("first cut", n, ctas);
    for (int c = 1; c <= n; ++c) {
        const int64_t x = share_start(U, n, c, ctas, step);
        if (U > 0 && (x <= before || (n > 1 && x - before < MIN_SHARE - 1)))
            return fail("cut", c, x - before);
        before = x;
    }
    if (before != U)
        return fail("last cut", before, U);
    return 0;
}

}  // namespace

int main()
{
    for (unsigned seed = 1; seed <= 400; ++seed)
        if (check_batch(seed))
            return 1;
    // lines far beyond 32 bits
    for (int ctas = 1; ctas < 300; ++ctas)
        for (int64_t U : {int64_t(1) << 33, (int64_t(1) << 40) + 12345, int64_t(4) * ctas}) {
            const int n = shares(U, ctas);
            int64_t before = 0;
            for (int c = 1; c <= n; ++c) {
                const int64_t x = share_start(U, n, c, ctas, share_step(ctas));
                if (x <= before || x > U)
                    return fail("long line", ctas, c);
                before = x;
            }
            if (before != U)
                return fail("long line's end", before, U);
        }
    std::printf("ok\n");
    return 0;
}
