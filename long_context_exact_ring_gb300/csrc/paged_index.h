// paged_index.h -- index arithmetic of the paged cache that device data
// decides and the host cannot check: which rows a request has, and where a
// key lies.  Plain C++, so that it is tested on the CPU as it runs on the
// GPU.
#pragma once

#ifdef __CUDACC__
#define RA_HD __host__ __device__ __forceinline__
#else
#define RA_HD inline
#endif

namespace ra {
namespace paged {

// A pool of pages: row (page, token, head) at page * sp + token * st +
// head * sh elements, its d elements contiguous.
struct PoolLayout {
    long long sp, st, sh;
};

// A request's first row of q, its new tokens and its keys.
struct Request {
    int first, q, len;
};

// From two neighbouring entries of cu_q and a length, cut to the `tokens`
// rows of q and the keys a table row can name.
RA_HD Request cut_request(int cu0, int cu1, int len, int tokens, int max_pages, int page_size)
{
    Request r;
    const long long capacity = (long long)max_pages * page_size;
    const int a = cu0 < 0 ? 0 : (cu0 > tokens ? tokens : cu0);
    const int b = cu1 < a ? a : (cu1 > tokens ? tokens : cu1);
    r.first = a;
    r.q = b - a;
    r.len = len < 0 ? 0 : (len > capacity ? (int)capacity : len);
    return r;
}

// Index of a key's page in its table row; page_shift >= 0 where page_size is
// 1 << page_shift.
RA_HD int page_index(int key, int page_size, int page_shift)
{
    return page_shift >= 0 ? key >> page_shift : key / page_size;
}

RA_HD bool page_ok(int page, int num_pages) { return (unsigned)page < (unsigned)num_pages; }

// Element offset of row (page, offset, head).
RA_HD long long row_offset(const PoolLayout& l, int page, int offset, int head)
{
    return page * l.sp + offset * l.st + head * l.sh;
}

// Block b's share of `total` units over `blocks` (at most 2^16) equal blocks:
// units [start, start + count).  Divides 16 bits at a time: a 64-bit division
// is a function call on the GPU.
struct Share {
    long long start, count;
};

RA_HD Share share_of(long long total, int blocks, int b)
{
    unsigned long long quotient = 0;
    unsigned rest = 0;
    for (int x = 48; x >= 0; x -= 16) {
        const unsigned part = rest << 16 | (unsigned)((unsigned long long)total >> x & 0xffffu);
        quotient = quotient << 16 | part / (unsigned)blocks;
        rest = part % (unsigned)blocks;
    }
    const long long each = (long long)quotient, over = (long long)rest;
    Share s;
    s.start = each * b + (b < over ? b : over);
    s.count = each + (b < over ? 1 : 0);
    return s;
}

// x / size of a quotient below `count`, by bisection.
RA_HD int quotient_below(long long x, long long size, int count)
{
    int lo = 0, hi = count;
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (mid * size <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// sum over i in [0, n) of floor((a i + b) / m), by Euclid's steps on (a, m).
// a n + b and the quotients' top values stay below 2^32.
RA_HD long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b)
{
    unsigned long long sum = 0;
    while (true) {
        const unsigned qa = a / m, qb = b / m;
        sum += (unsigned long long)n * (n - 1) / 2 * qa + (unsigned long long)n * qb;
        a -= qa * m;
        b -= qb * m;
        const unsigned top = a * n + b;
        if (top < m) return (long long)sum;
        n = top / m;
        b = top - n * m;
        const unsigned x = a;
        a = m;
        m = x;
    }
}

// A request's tiles of `step` new tokens and what they cost: the steps of
// `unit` keys up to the last key that the tile's last token sees, at least
// one, and `extra` of them for beginning and ending a tile.
struct TileWork {
    int q, len, causal, step, unit, extra;

    RA_HD int tiles() const { return (q + step - 1) / step; }
    // keys that tile t's last token sees
    RA_HD int keys(int t) const
    {
        if (!causal) return len;
        const long long end = (long long)(t + 1) * step;
        const int seen = len - q + (int)(end < q ? end : q);
        return seen > 0 ? seen : 0;
    }
    RA_HD int units(int t) const
    {
        const int k = keys(t);
        return k > 0 ? (k + unit - 1) / unit : 1;
    }
    // cost of the tiles before t, 0 <= t <= tiles()
    RA_HD long long before(int t) const
    {
        if (t <= 0) return 0;
        long long sum = (long long)t * extra;
        if (!causal) return sum + (long long)t * units(0);
        // the last tile may be short: it comes on top
        if (t == tiles()) sum += units(--t);
        // tiles 0 .. t-1 end at token (i + 1) step: units 1 + (first + i step) / unit
        // from the first tile on that sees a key
        const int first = len - q + step - 1;
        const int blind = first < 0 ? (-first + step - 1) / step : 0;
        sum += t;
        if (t <= blind) return sum;
        return sum + floor_sum((unsigned)(t - blind), (unsigned)unit, (unsigned)step, (unsigned)(first + blind * step));
    }
    // the tile that cost x lies in, out of tiles [lo, hi), before(lo) <= x < before(hi)
    RA_HD int tile_of(long long x, int lo, int hi) const
    {
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before(mid) <= x) lo = mid;
            else hi = mid;
        }
        return lo;
    }
};

// Where a share's end at cost `c` cuts a tile: the steps of keys in front of
// it.  A tile's extra cost comes first, so a cut inside it is one in front of
// the tile.
RA_HD int cut_units(long long c, int extra) { return c > extra ? (int)(c - extra) : 0; }

}  // namespace paged
}  // namespace ra
