// paged_cache.cuh -- the bookkeeping of a paged key/value cache:
//   paged_plan_kernel    pages, slots and lengths of the next step
//   paged_append_kernel  new K and V rows into the pool
#pragma once

#include "paged_index.h"
#include "sm103_ptx.cuh"

namespace ra {
namespace paged {

constexpr int kMaxRequests = 8192;
constexpr int kPlanThreads = 1024;

// One step's bookkeeping.  With pages(x) = ceil(x / page_size), request i
// of len_i cached tokens and new_i more:
//   released pages   r_i = pages(len_i) if new_i < 0, else 0
//   A                F + sum r, F = counts[0], the stack's height
//   cu_q             exclusive sums of max(new_i, 0)
//   need_i           pages(len_i + new_i) - pages(len_i), N_i its exclusive sums
//   granted_i        need_i = 0, or N_i + need_i <= A
//   k-th new page    stack[A - 1 - (N_i + k)]
// where stack[x] is free_list[x] below F and the released pages, in order,
// above.  The stack is never popped in memory, only in the count, so every
// entry read was there before the call and no thread waits for another's
// store.
//
// A latency problem: three block scans over the requests, then independent
// stores.  One block; the requests' sums stay in shared memory and the
// stores find their request by bisection.
struct PlanParams {
    const int* seq_lens;
    const int* new_lens;
    int* table;
    long long table_stride;
    int* free_list;
    const int* counts;
    int* seq_out;
    int* cu_q;
    int* slots;
    int* counts_out;
    int n, max_pages, num_pages, page_size, tokens;
};

// Shared memory of a plan over n requests: four int arrays.
__host__ __device__ constexpr size_t plan_smem(int n) { return (size_t)(4 * (n + 1)) * sizeof(int); }

// Exclusive sum over the block; *total receives the whole sum.  Every thread
// calls it; `scratch` holds one value per warp and one more.
__device__ __forceinline__ long long block_exclusive_sum(long long v, long long* scratch, long long* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    if (warp == 0) {
        long long s = lane < warps ? scratch[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        if (lane < warps) scratch[lane] = s;
    }
    __syncthreads();
    *total = scratch[warps - 1];
    return x - v + (warp ? scratch[warp - 1] : 0);
}

// Largest i in [0, n) with a[i] <= x, given a[0] <= x (a is nondecreasing;
// among equal entries the last, the one that is not empty).
__device__ __forceinline__ int find_last_le(const int* a, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PlanParams p)
{
    extern __shared__ int plan_smem_raw[];
    __shared__ long long scratch[33];
    int* s_cu = plan_smem_raw;              // [n + 1] exclusive sums of the new tokens
    int* s_take = s_cu + (p.n + 1);         // [n + 1] exclusive sums of the granted pages
    int* s_rel = s_take + (p.n + 1);        // [n + 1] exclusive sums of the released pages
    int* s_len = s_rel + (p.n + 1);         // [n] cached tokens, or ~tokens if not granted
    const int tid = threadIdx.x, n = p.n, ps = p.page_size;
    const long long capacity = (long long)p.max_pages * ps;
    const int per = (n + kPlanThreads - 1) / kPlanThreads;
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    auto pages = [&](long long x) { return (x + ps - 1) / ps; };
    auto length = [&](int i) { return min((long long)max(p.seq_lens[i], 0), capacity); };

    const int F = min(max(p.counts[0], 0), p.num_pages);
    long long add = 0, rel = 0;
    for (int i = i0; i < i1; ++i) {
        const int q = p.new_lens[i];
        if (q < 0) rel += pages(length(i));
        else add += q;
    }
    long long add_total, rel_total, need_total;
    const long long add0 = block_exclusive_sum(add, scratch, &add_total);
    const long long rel0 = block_exclusive_sum(rel, scratch, &rel_total);
    const long long A = F + rel_total;
    // pages the request would need: 0 if it cannot fit its table row or the slots
    auto need_of = [&](int i, long long cu, bool* fits) {
        const int q = p.new_lens[i];
        const long long len = length(i);
        const long long after = pages(len + max(q, 0));
        *fits = q >= 0 && after <= p.max_pages && cu + q <= p.tokens;
        return *fits ? after - pages(len) : 0ll;
    };
    long long need = 0, cu = add0;
    for (int i = i0; i < i1; ++i) {
        bool fits;
        need += need_of(i, cu, &fits);
        cu += max(p.new_lens[i], 0);
    }
    const long long need0 = block_exclusive_sum(need, scratch, &need_total);
    long long before = need0, released = rel0;
    int refused = 0;
    cu = add0;
    for (int i = i0; i < i1; ++i) {
        bool fits;
        const int q = p.new_lens[i];
        const long long len = length(i);
        const long long want = need_of(i, cu, &fits);
        const bool granted = fits && (want == 0 || before + want <= A);
        s_cu[i] = (int)min(cu, (long long)INT_MAX);
        s_take[i] = (int)min(before, A);     // requests past A get nothing
        s_rel[i] = (int)released;
        s_len[i] = granted ? (int)len : ~(int)len;
        refused += q >= 0 && !granted;
        before += want;
        cu += max(q, 0);
        if (q < 0) released += pages(len);
    }
    // pages handed out: all that were needed, or those of the granted prefix
    long long refused_total, taken_total;
    block_exclusive_sum(refused, scratch, &refused_total);
    {
        long long taken = 0, b = need0, c = add0;
        for (int i = i0; i < i1; ++i) {
            bool fits;
            const long long want = need_of(i, c, &fits);
            if (fits && b + want <= A) taken += want;
            b += want;
            c += max(p.new_lens[i], 0);
        }
        block_exclusive_sum(taken, scratch, &taken_total);
    }
    if (tid == 0) {
        s_cu[n] = (int)min(add_total, (long long)INT_MAX);
        s_take[n] = (int)min(need_total, A);
        s_rel[n] = (int)rel_total;
    }
    __syncthreads();   // every input length and count is read: outputs may alias them

    // A page of the stack, as it stands after the releases.
    auto stack = [&](int x) {
        if (x < F) return p.free_list[x];
        const int j = find_last_le(s_rel, n, x - F);
        return p.table[j * p.table_stride + (x - F - s_rel[j])];
    };
    for (int i = tid; i < n; i += kPlanThreads) {
        const int q = p.new_lens[i], l = s_len[i];
        const int len = l < 0 ? ~l : l;
        p.seq_out[i] = q < 0 ? 0 : (l < 0 ? len : len + q);
        p.cu_q[i] = s_cu[i];
    }
    if (tid == 0) {
        p.cu_q[n] = s_cu[n];
        p.counts_out[0] = (int)min(A - taken_total, (long long)p.num_pages);
        p.counts_out[1] = (int)refused_total;
    }
    for (int k = tid; k < (int)min(rel_total, (long long)p.num_pages - F); k += kPlanThreads) {
        const int j = find_last_le(s_rel, n, k);
        p.free_list[F + k] = p.table[j * p.table_stride + (k - s_rel[j])];
    }
    for (int k = tid; k < (int)taken_total; k += kPlanThreads) {
        const int i = find_last_le(s_take, n, k);
        p.table[i * p.table_stride + (int)pages(s_len[i]) + (k - s_take[i])] = stack((int)A - 1 - k);
    }
    for (int t = tid; t < p.tokens; t += kPlanThreads) {
        int slot = -1;
        if (t < s_cu[n]) {
            const int i = find_last_le(s_cu, n, t);
            const int len = s_len[i];
            if (len >= 0) {
                const int pos = len + (t - s_cu[i]);
                const int page_index = pos / ps, have = (int)pages(len);
                const int page = page_index < have ? p.table[i * p.table_stride + page_index]
                                                   : stack((int)A - 1 - (s_take[i] + page_index - have));
                if (page_ok(page, p.num_pages)) slot = page * ps + (pos - page_index * ps);
            }
        }
        p.slots[t] = slot;
    }
}

// K and V rows of the new tokens to their slots; every thread moves 16 bytes
// of each.  Bound by HBM (four bytes moved for each two of a row) or, for a
// decode step's few tokens, by the launch.
__global__ void __launch_bounds__(256)
paged_append_kernel(const uint16_t* __restrict__ k, long long k_tok, long long k_head,
                    const uint16_t* __restrict__ v, long long v_tok, long long v_head, uint16_t* __restrict__ kc,
                    PoolLayout lk, uint16_t* __restrict__ vc, PoolLayout lv, const int* __restrict__ slots,
                    int tokens, int heads, int vec_shift, int page_size, int num_slots, uint32_t* status)
{
    const uint32_t per_token = (uint32_t)heads << vec_shift;      // 16-byte pieces of a token's K
    const uint64_t total = (uint64_t)tokens * per_token;
    for (uint64_t x = (uint64_t)blockIdx.x * 256 + threadIdx.x; x < total; x += (uint64_t)gridDim.x * 256) {
        const uint32_t t = (uint32_t)(x / per_token);
        const uint32_t piece = (uint32_t)(x - (uint64_t)t * per_token);
        const uint32_t h = piece >> vec_shift, e = (piece & ((1u << vec_shift) - 1u)) * 8u;
        const int slot = slots[t];
        if ((unsigned)slot >= (unsigned)num_slots) {
            if (slot != -1) atomicOr(status, kStatusBadPage);
            continue;
        }
        const uint4 a = *reinterpret_cast<const uint4*>(k + t * k_tok + h * k_head + e);
        const uint4 b = *reinterpret_cast<const uint4*>(v + t * v_tok + h * v_head + e);
        const int page = slot / page_size, off = slot - page * page_size;
        *reinterpret_cast<uint4*>(kc + row_offset(lk, page, off, h) + e) = a;
        *reinterpret_cast<uint4*>(vc + row_offset(lv, page, off, h) + e) = b;
    }
}

}  // namespace paged
}  // namespace ra
