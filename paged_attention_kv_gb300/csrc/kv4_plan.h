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

// What a key costs with so many rows beside it, and an item by itself (its start,
// which is a chain of trips to memory, and its end): as much as so many keys. 100
// requests of 1 to 15 tokens and 500 to 2000 keys: 104.9 us, 109.5 with 11 in place
// of 9, 113.5 with 7 and 12, 103.5 with one weight for all, which costs 256 requests
// of 1 to 8 tokens 138.9 us against 130.1. Items at 48 keys instead of 96: two short
// requests 6.7 us instead of 5.0, 128 requests of 4 tokens and 30 to 2000 keys 46.1
// instead of 40.0; at 192 those take 41.5.
PKV_HD int kv4_weight(int rows) { return rows <= 8 ? 4 : rows <= 16 ? 6 : 9; }
constexpr int kKv4ItemKeys = 96;

// About x / y (2^-21), in a few cycles on the device: every warp works its share out
// before it can ask for any key.
PKV_HD float kv4_ratio(float x, float y) {
#ifdef __CUDA_ARCH__
    return __fdividef(x, y);
#else
    return x / y;
#endif
}
// x / y for a quotient below 2^19, without a division of 64 bits.
PKV_HD int kv4_quotient(long long x, long long y) {
    int q = (int)kv4_ratio((float)x, (float)y);  // off by at most 1
    const long long left = x - q * y;
    if (left < 0) --q;
    if (left >= y) ++q;
    return q;
}

PKV_HD Kv4Request kv4_request(int q0, int n, int len, int group, int rows) {
    Kv4Request q{q0, n, len, 0, 0, 0};
    const unsigned all = (unsigned)n * (unsigned)group;  // below 2^31
    q.tiles = (int)((all + (unsigned)rows - 1) / (unsigned)rows);
    if (q.tiles <= 1) {
        q.c0 = (long long)kv4_weight((int)all) * ((long long)len + kKv4ItemKeys);
    } else {
        const int step = kv4_weight(rows) * rows / group;  // keys more from tile to tile
        q.c0 = (long long)kv4_weight(rows) * ((long long)len - n + kKv4ItemKeys) + step;
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
        const int mid = lo + (hi - lo + 1) / 2;
        if (kv4_cost(q, heads, mid) <= off) lo = mid; else hi = mid - 1;
    }
    const long long first = kv4_cost(q, heads, lo), c = kv4_item_cost(q, lo);
    *i = lo;
    *h = kv4_quotient(off - first, c);
    *start = first + *h * c;
}

PKV_HD Kv4Tiling kv4_tile(const Kv4Request &q, int i, int group, int rows) {
    const unsigned from = (unsigned)i * (unsigned)rows, left = (unsigned)q.n * (unsigned)group - from;
    Kv4Tiling t;
    t.rows = left < (unsigned)rows ? (int)left : rows;
    t.keys = q.tiles == 1 ? q.len : q.len - q.n + (int)((from + t.rows - 1) / (unsigned)group) + 1;
    t.blocks = (int)(((unsigned)t.keys + 15) / 16);
    return t;
}

// The block before which an item is cut at its position `off`, with so many blocks
// a position: an even one (a warp
// takes two at a time), none and all of them included, so that no piece is
// shorter than two. Both shares that meet there work it out alike, and it does
// not fall as off rises.
PKV_HD int kv4_cut(long long off, float each, int blocks) {
    const int b = (int)((float)off * each) & ~1;
    return b + 2 > blocks ? blocks : b;
}

// Requests of the chunk kernel: tiles of 128 rows, keys in tiles of 128. Half a tile
// is worth it: 64 rows of 64 requests with 1000 keys take 61 us there, 110 here.
constexpr int kKv4ChunkRows = 128;
PKV_HD bool kv4_is_chunk(const Kv4Request &q, int group) { return (long long)q.n * group >= 64; }
PKV_HD int kv4_chunk_tiles(int keys) { return (int)(((unsigned)keys + 127) / 128); }
// Its key tiles of all heads, about (q made with tiles of 128 rows).
PKV_HD long long kv4_chunk_units(const Kv4Request &q, int heads) {
    return (long long)q.tiles * heads * kv4_chunk_tiles(q.len - q.n / 2);
}
// Where the chunk kernel's items leave CTAs idle, each is split by keys into as many
// parts as there are CTAs for it (two an SM), of four key tiles at least, of ten where
// most items have an SM to themselves as it is. Split and not: 4 requests of 64 tokens
// and 4000 keys (8 heads of 128) 42 and 60 us, 1 of 512 and 30000 279 and 394; 16 of 32
// and 2000, whose parts would have eight, 43 and 40.
struct Kv4Splits {
    int count, least;  // parts of an item at most, key tiles of a part at least (4 or 10)
};
constexpr int kKv4MaxSplits = 8;
PKV_HD Kv4Splits kv4_splits(long long items, int sms) {
    if (items <= 0 || items > sms) return Kv4Splits{1, 4};
    const int n = kv4_quotient(2 * sms, items);
    return Kv4Splits{n < kKv4MaxSplits ? n : kKv4MaxSplits, n < 4 ? 10 : 4};
}
// In how many parts so many key tiles are, and where part s begins.
PKV_HD int kv4_parts(int tiles, Kv4Splits sp) {
    const int n = sp.least == 4 ? tiles / 4 : tiles / 10;
    return n < 2 ? 1 : n < sp.count ? n : sp.count;
}
PKV_HD int kv4_part_begin(int tiles, int parts, int s) { return (int)((unsigned)(tiles * s) / (unsigned)parts); }  // 8 * 2^24 at most

// Which kernel has them. The chunk kernel takes about 7 us and 1.4 to 1.7 a key tile of
// the longest part. The other one cuts items into equal shares: about 20 us and 20 to
// 30 ns for each of all units. Measured (this kernel, the other): 1 request of 32 tokens
// and 1000 keys of 8 heads of 128 22.5 and 35 us, 16000 keys 46 and 61; 16 of 16 tokens
// and 4000 keys 64 and 96; 1 of 512 tokens and 30000 keys 279 and 831; 1 of 64 tokens and
// 60000 keys of 2 heads of 128 116 and 131.
PKV_HD bool kv4_use_chunks(long long units, int longest, Kv4Splits sp) {
    return units > 0 && (units + 400) * kv4_parts(longest, sp) >= 48LL * longest;
}

struct Kv4Shares {
    long long total, each;
    int count, per_cta;  // shares; of one CTA: CTA c has shares c * per_cta on

    PKV_HD long long begin(int k) const { return k < count ? k * each : total; }
    // the share that a position lies in
    PKV_HD int index(long long pos) const { return kv4_quotient(pos, each); }
};

// Share k's piece [b0, b1) of the item that starts at `start`.
struct Kv4Piece {
    int b0, b1;
    bool begun, cut, more;  // it begins in a share before, ends in one behind; the share goes on behind the item
    int first, last;        // the shares that hold pieces of it
};
PKV_HD Kv4Piece kv4_piece(const Kv4Shares &sh, int k, long long start, long long cost, int blocks) {
    const long long from = sh.begin(k), to = sh.begin(k + 1), stop = start + cost;
    const float each = kv4_ratio((float)blocks, (float)cost);
    Kv4Piece p;
    p.b0 = from > start ? kv4_cut(from - start, each, blocks) : 0;
    p.b1 = to < stop ? kv4_cut(to - start, each, blocks) : blocks;
    p.begun = p.b0 > 0;
    p.cut = p.b1 < blocks;
    p.more = stop < to;
    p.first = p.last = k;
    // a cut that moved to the item's start or end takes its share out (only one can:
    // shares are longer than two blocks)
    if (p.begun) {
        p.first = sh.index(start);
        if (kv4_cut(sh.begin(p.first + 1) - start, each, blocks) == 0) ++p.first;
    }
    if (p.cut) {
        p.last = sh.index(stop - 1);
        if (kv4_cut(sh.begin(p.last) - start, each, blocks) == blocks) --p.last;
    }
    return p;
}

// What a share has at least: six blocks of the rows of a tile. An item that is cut
// has four blocks or more, and costs kKv4ItemKeys / 16 = 6 more than those, so that
// a share holds more than two of its blocks: see kv4_piece. (Ten blocks: two short
// requests 6.6 us instead of 5.0, 8 of 500 to 2000 keys 14.4 instead of 12.7.)
PKV_HD int kv4_least(int rows) { return 6 * 16 * kv4_weight(rows); }

// At most ctas * warps shares of at least `least`. Where that leaves warps idle, up to
// six shares of an item (of the mean of `reqs` requests' kv heads) go into one CTA: it
// joins them in 1 us, where parts of other CTAs take 3. The kv heads of a request alone
// are of one length and get shares that end where they do.
PKV_HD Kv4Shares kv4_shares(long long total, int ctas, int warps, int least, int reqs, int heads) {
    const int most = ctas * warps;
    Kv4Shares s;
    s.total = total;
    int together = 0;
    if (total <= 0) {
        s.each = least;
    } else if (total <= (long long)least * most) {
        const float mean = kv4_ratio((float)total, (float)reqs * (float)heads);
        const int k = (int)kv4_ratio(mean, (float)least);
        s.each = reqs == 1 && k > 1 ? (total / heads + k - 1) / k : least;
        together = k < 6 ? k : 6;
    } else {
        s.each = (long long)(kv4_ratio((float)total, (float)most) * 1.000001f) + 1;
        while (s.each * most < total) s.each += 1 + (s.each >> 22);
    }
    s.count = total <= 0 ? 0 : kv4_quotient(total - 1, s.each) + 1;
    s.per_cta = kv4_quotient(s.count + ctas - 1, ctas);
    if (s.per_cta < together) s.per_cta = together < warps ? together : warps;
    return s;
}

}  // namespace pkv
