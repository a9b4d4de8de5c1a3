// How paged_chunk_attention's work is cut into one share a CTA.
//
// An item is a row tile of one (sequence, KV head): up to `rows` (token, query head)
// rows, tpr = rows / G tokens of all G query heads of the KV head.  It covers the key
// tiles (of 128) from the first that its first token sees to the last that its last
// one does.  Items are numbered by sequence, KV head, row tile; an item costs its tiles
// and ITEM_COST more for its q, its first tile's latency and its output.  (A tile counts the
// same whatever rows the item has: shares of batches of long pieces and single tokens are
// equal in tiles, not in time.)  The costs end
// to end are a line that is cut into equal shares; a cut within an item falls between two of its
// tiles.  Where a position of the line falls is worked out in closed form, so a CTA
// finds its share without looking at other CTAs' items.  Host and device.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define PKV_HD __host__ __device__ __forceinline__
#else
#define PKV_HD inline
#endif

namespace pkv {
namespace chunk {

constexpr int TILE = 128, LG_TILE = 7;   // keys of a tile
// Measured with 0, 1, 2 and 4: 768 items of up to 16 tiles 91, 73, 66, 66 us; whole prompts 474,
// 449, 443, 452; drafts, one long sequence, pieces and windows the same within 2%.
constexpr int ITEM_COST = 2;

struct Rules {
    int lg_tpr;                       // tokens of a row tile: tpr = 2^lg_tpr, 16..256
    int window;                       // 0: none
    bool tree;                        // every new token may see any other
};

// sum over s < x of floor((a + s w) / 128), w = 2^lg_w, a >= 0.  (Shifts: a division of 64-bit
// integers is a hundred instructions.)
PKV_HD int64_t floor_sum(int64_t x, int64_t a, int lg_w)
{
    if (lg_w >= LG_TILE)
        return x * (a >> LG_TILE) + ((x * (x - 1) / 2) << (lg_w - LG_TILE));
    const int lg_k = LG_TILE - lg_w;
    // floor((a + s w) / 128) = floor((floor(a / w) + s) / k), k = 128 / w; H(y) sums floor(i / k)
    // over i < y: k q (q - 1) / 2 + (y - q k) q with q = floor(y / k)
    const int64_t y0 = a >> lg_w, y1 = y0 + x, q0 = y0 >> lg_k, q1 = y1 >> lg_k;
    const int64_t h0 = ((q0 * (q0 - 1) / 2) << lg_k) + (y0 - (q0 << lg_k)) * q0;
    const int64_t h1 = ((q1 * (q1 - 1) / 2) << lg_k) + (y1 - (q1 << lg_k)) * q1;
    return h1 - h0;
}

// One sequence: n new tokens, the last of L cached rows (0 < n <= L).
struct Seq {
    int n, L;
};

PKV_HD int row_tiles(const Rules &r, const Seq &q) { return ((q.n - 1) >> r.lg_tpr) + 1; }

// Positions of a row tile's first token and of the last key that a row of it may see.
PKV_HD void span(const Rules &r, const Seq &q, int rt, int &first, int &last)
{
    const int at = rt << r.lg_tpr, tpr = 1 << r.lg_tpr, end = q.n - at < tpr ? q.n : at + tpr;
    first = q.L - q.n + at;
    last = (r.tree ? q.L : q.L - q.n + end) - 1;
}

// Its key tiles [lo, hi).
PKV_HD void tiles(const Rules &r, const Seq &q, int rt, int &lo, int &hi)
{
    int first, last;
    span(r, q, rt, first, last);
    lo = r.window > 0 && first - r.window + 1 > 0 ? (first - r.window + 1) >> LG_TILE : 0;
    hi = (last >> LG_TILE) + 1;
}

// Cost of the row tiles before rt, all of them whole ones (of one KV head).
PKV_HD int64_t cost_before(const Rules &r, const Seq &q, int64_t rt)
{
    const int64_t A = q.L - q.n, tpr = 1 << r.lg_tpr;
    if (r.tree)
        return rt * (((q.L - 1) >> LG_TILE) + 1 + ITEM_COST);
    int64_t c = floor_sum(rt, A + tpr - 1, r.lg_tpr) + rt * (1 + ITEM_COST);
    if (r.window > 0) {
        const int64_t first = A - r.window + 1;
        const int64_t s0 = first < 0 ? (-first + tpr - 1) >> r.lg_tpr : 0;   // tiles from key 0
        if (rt > s0)
            c -= floor_sum(rt - s0, first + (s0 << r.lg_tpr), r.lg_tpr);
    }
    return c;
}

PKV_HD int64_t cost_of(const Rules &r, const Seq &q)
{
    const int R = row_tiles(r, q);
    int lo, hi;
    tiles(r, q, R - 1, lo, hi);
    return cost_before(r, q, R - 1) + (hi - lo) + ITEM_COST;
}

// A place between two tiles: of sequence b, KV head h, row tile rt, before key tile
// `tile`; `split`: within the item, not at its start.
struct Place {
    int b, h, rt, tile, split;
};

// Position x (0 <= x < Hkv * c, c the sequence's cost_of) of sequence b's stretch of the line.
PKV_HD Place place_in(const Rules &r, const Seq &q, int b, int64_t x, int64_t c)
{
    Place p;
    p.b = b;
    // x / c, by an estimate that is put right (a division of 64-bit integers is a hundred
    // instructions, and the start of a kernel waits for all of those that it runs)
    int64_t h = (int64_t)((float)x / (float)c);
    while (h * c > x)
        --h;
    while ((h + 1) * c <= x)
        ++h;
    p.h = (int)h;
    x -= h * c;
    int a = 0, e = row_tiles(r, q) - 1;               // the last row tile that starts by x
    int64_t before = 0;                               // and the cost before it
    while (a < e) {
        const int m = (a + e + 1) / 2;
        const int64_t cm = cost_before(r, q, m);
        if (cm <= x) {
            a = m;
            before = cm;
        } else {
            e = m - 1;
        }
    }
    p.rt = a;
    x -= before;
    int lo, hi;
    tiles(r, q, a, lo, hi);
    p.tile = x > ITEM_COST ? lo + (int)(x - ITEM_COST) : lo;
    p.split = p.tile > lo;
    return p;
}

// Shares for a line of length U on `ctas` CTAs: equal ones, but none shorter than MIN_SHARE
// (a share of a tile or two costs more in its start and in the joining of its state
// than it saves).  Measured with 2, 4, 8 and 16: 8 tokens of 8 KV heads over 500 rows 13.2, 14.4, 17.9,
// 24.2 us, over 2000 rows 16.8, 16.3, 18.8, 24.9, over 8000 rows 27.5, 24.4, 22.0, 32.0; calls
// whose shares are longer anyway are the same.
constexpr int MIN_SHARE = 4;
PKV_HD int shares(int64_t U, int ctas)
{
    return U >= (int64_t)MIN_SHARE * ctas ? ctas : U < MIN_SHARE ? 1 : (int)(U / MIN_SHARE);
}
// 2^32 / ctas, rounded up: what share_start multiplies by instead of dividing.
inline uint32_t share_step(int ctas) { return (uint32_t)((((uint64_t)1 << 32) + ctas - 1) / ctas); }

// Where share c of n (or the line's end, c = n) starts.
PKV_HD int64_t share_start(int64_t U, int n, int c, int ctas, uint32_t step)
{
    if (c >= n)
        return U;
    if (n < ctas)
        return (int64_t)c * MIN_SHARE;
    // U c step / 2^32: the product c step is below 2^32 for c < ctas
    const uint64_t f = (uint64_t)c * step;
#if defined(__CUDA_ARCH__)
    return (int64_t)__umul64hi((uint64_t)U, f << 32);
#else
    return (int64_t)(((unsigned __int128)(uint64_t)U * f) >> 32);
#endif
}

// What a share does of an item.
struct Piece {
    int b, h;
    int tok;               // first token, as a row of q
    int rows;
    int first, last;       // positions of the first token and of the last key in sight
    int sight;             // first key in sight of any row
    int base;              // cached rows before the new tokens (L - n)
    int len;               // L
    int t0, t1;            // key tiles
    int kind;              // 0: the whole item; 1: not from its start; 2: from its start, not to its end;
                           // -1: no more pieces
};

// A share's walk over its items' pieces.  `lengths(b, q, q0)`: sequence b's, and its first token
// as a row of q; false if it has no work.
struct Walk {
    Place at, end;
    Seq q;
    int q0;

    template <typename F>
    PKV_HD void start(int batch, const Place *places, F lengths)
    {
        at = places[0];
        end = places[1];
        if (at.b < batch)
            lengths(at.b, q, q0);
    }

    template <typename F>
    PKV_HD bool next(const Rules &r, int batch, int num_kv_heads, int lg_g, Piece &c, F lengths)
    {
        const bool last_item = at.b == end.b && at.h == end.h && at.rt == end.rt;
        if (at.b >= batch || (last_item && at.tile >= end.tile))
            return false;
        const int tok = at.rt << r.lg_tpr, tpr = 1 << r.lg_tpr;
        int lo, hi;
        tiles(r, q, at.rt, lo, hi);
        span(r, q, at.rt, c.first, c.last);
        c.b = at.b;
        c.h = at.h;
        c.tok = q0 + tok;
        c.rows = (q.n - tok < tpr ? q.n - tok : tpr) << lg_g;
        c.sight = r.window > 0 && c.first - r.window + 1 > 0 ? c.first - r.window + 1 : 0;
        c.base = q.L - q.n;
        c.len = q.L;
        c.t0 = at.tile;
        c.t1 = last_item ? end.tile : hi;
        c.kind = c.t0 > lo ? 1 : c.t1 < hi ? 2 : 0;
        if (last_item) {
            at.tile = end.tile;
            return true;
        }
        if (++at.rt == row_tiles(r, q)) {
            at.rt = 0;
            if (++at.h == num_kv_heads) {
                at.h = 0;
                do
                    ++at.b;
                while (at.b < batch && !lengths(at.b, q, q0));
                if (at.b >= batch)
                    return true;
            }
        }
        tiles(r, q, at.rt, lo, hi);
        at.tile = lo;
        return true;
    }
};

// Share c starts within an item, at place `a` (a.split): how many pieces the item has if c is the
// first share to start within it, else 0.  Its first piece is then share c - 1's last, the others
// the first ones of shares c, c + 1, ..  (A share leaves at most two states: that of its
// first piece, kind 1, and that of its last, kind 2.)
PKV_HD int pieces_to_join(const Rules &r, const Seq &q, const Place &a, int64_t U, int n, int c,
                          int ctas, uint32_t step)
{
    int lo, hi;
    tiles(r, q, a.rt, lo, hi);
    // positions on the line: where the item may first be cut, and its end
    const int64_t first = share_start(U, n, c, ctas, step) - (a.tile - lo), end = first + (hi - lo);
    if (share_start(U, n, c - 1, ctas, step) > first)
        return 0;
    int pieces = 2;
    while (c + pieces - 1 < n && share_start(U, n, c + pieces - 1, ctas, step) < end)
        ++pieces;
    return pieces;
}

}  // namespace chunk
}  // namespace pkv
