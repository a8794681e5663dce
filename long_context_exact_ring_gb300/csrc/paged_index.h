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

// sum over i in [0, n) of floor((a i + b) / m), by Euclid's steps on (a, m).
RA_HD long long floor_sum(unsigned long long n, unsigned long long m, unsigned long long a, unsigned long long b)
{
    unsigned long long sum = 0;
    while (true) {
        sum += n * (n - 1) / 2 * (a / m) + n * (b / m);
        a %= m;
        b %= m;
        const unsigned long long top = a * n + b;
        if (top < m) return (long long)sum;
        n = top / m;
        b = top % m;
        const unsigned long long x = a;
        a = m;
        m = x;
    }
}

// A request's tiles of `step` new tokens, and the steps of `unit` keys that
// each takes: those up to the last key its last token sees, at least one.
struct TileWork {
    int q, len, causal, step, unit;

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
    // units of the tiles before t, 0 <= t <= tiles()
    RA_HD long long before(int t) const
    {
        if (t <= 0) return 0;
        if (!causal) return (long long)t * units(0);
        if (t == tiles()) return before(t - 1) + units(t - 1);
        // tiles 0 .. t-1 end at token (i + 1) step: units 1 + (first + i step) / unit
        // from the first tile on that sees a key
        const long long first = (long long)len - q + step - 1;
        const long long blind = first < 0 ? (-first + step - 1) / step : 0;
        if (t <= blind) return t;
        return t + floor_sum((unsigned long long)(t - blind), (unsigned long long)unit, (unsigned long long)step,
                             (unsigned long long)(first + blind * step));
    }
    // the tile that unit x of the request's tiles lies in, 0 <= x < before(tiles())
    RA_HD int tile_of(long long x) const
    {
        int lo = 0, hi = tiles();
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before(mid) <= x) lo = mid;
            else hi = mid;
        }
        return lo;
    }
};

}  // namespace paged
}  // namespace ra
