// How attention over the 4-bit pool is cut into equal shares, on the host and
// on the device alike.
//
// A request with n queries and `len` keys has n * group rows of a kv head, in
// tiles of `rows`; an item is (request, tile, kv head), in that order, and costs
// its keys times a weight of its rows. All items of the batch in a row are cut
// into equal shares, one a warp, whatever items they cut through. Costs only
// balance the shares: any rule gives right results, so a long request's tiles
// get costs that rise by a constant, whose sums need no loop.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define PKV_HD __host__ __device__ __forceinline__
#else
#define PKV_HD inline
#endif

namespace pkv {

struct Kv4Request {
    int q0, n, len;     // first token of the batch, queries, keys
    int tiles;          // of each kv head; 0: nothing to do
    long long c0, c1;   // item i of a kv head costs c0 + i * c1
};

struct Kv4Tiling {
    int rows, keys, blocks;  // rows of the tile, keys its last row sees, blocks of those
};

// What a key costs with so many rows beside it, and what an item costs by itself
// (start, end, partials), as a number of keys of weight 1.
PKV_HD int kv4_weight(int rows) { return rows <= 8 ? 4 : rows <= 16 ? 6 : 11; }
constexpr int kKv4ItemCost = 128;

PKV_HD Kv4Request kv4_request(int q0, int n, int len, int group, int rows) {
    Kv4Request q{q0, n, len, 0, 0, 0};
    const long long all = (long long)n * group;
    q.tiles = (int)((all + rows - 1) / rows);
    if (q.tiles <= 1) {
        q.c0 = (long long)kv4_weight((int)all) * len + kKv4ItemCost;
    } else {
        const long long step = (long long)kv4_weight(rows) * rows / group;  // keys more from tile to tile
        q.c0 = (long long)kv4_weight(rows) * (len - n) + step + kKv4ItemCost;
        q.c1 = step;
    }
    return q;
}

// Of the first `upto` tiles.
PKV_HD long long kv4_cost(const Kv4Request &q, int heads, long long upto) {
    return heads * (upto * q.c0 + q.c1 * (upto * (upto - 1) / 2));
}
PKV_HD long long kv4_item_cost(const Kv4Request &q, int i) { return q.c0 + i * q.c1; }

// The item that position `off` of a request lies in, and that item's first position.
PKV_HD void kv4_locate(const Kv4Request &q, int heads, long long off, int *i, int *h, long long *start) {
    int lo = 0, hi = q.tiles - 1;  // the last tile that starts at or before off
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (kv4_cost(q, heads, mid) <= off) lo = mid; else hi = mid - 1;
    }
    const long long first = kv4_cost(q, heads, lo), c = kv4_item_cost(q, lo);
    *i = lo;
    *h = (int)((off - first) / c);
    *start = first + *h * c;
}

PKV_HD Kv4Tiling kv4_tile(const Kv4Request &q, int i, int group, int rows) {
    const long long left = (long long)q.n * group - (long long)i * rows;
    Kv4Tiling t;
    t.rows = left < rows ? (int)left : rows;
    t.keys = q.len - q.n + (int)(((long long)i * rows + t.rows - 1) / group) + 1;
    t.blocks = (t.keys + 15) / 16;
    return t;
}

// The block at which position `off` of an item of this cost lies.
PKV_HD int kv4_block_at(long long off, long long cost, int blocks) { return (int)(off * blocks / cost); }

struct Kv4Shares {
    int count;
    long long total, each, rest;

    PKV_HD long long begin(int k) const { return each * k + rest * k / count; }
    // the share that a position lies in
    PKV_HD int index(long long pos) const {
        int k = (int)((double)pos / (double)total * count);
        k = k < 0 ? 0 : k >= count ? count - 1 : k;
        while (k + 1 < count && begin(k + 1) <= pos) ++k;
        while (k > 0 && begin(k) > pos) --k;
        return k;
    }
};

// At most `most` shares of at least `least`.
PKV_HD Kv4Shares kv4_shares(long long total, int most, int least) {
    Kv4Shares s;
    s.total = total;
    s.count = total <= 0 ? 0 : total / least < 1 ? 1 : total / least > most ? most : (int)(total / least);
    s.each = s.count ? total / s.count : 0;
    s.rest = s.count ? total % s.count : 0;
    return s;
}

}  // namespace pkv
