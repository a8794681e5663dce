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

}  // namespace paged
}  // namespace ra
