// paged_cache.cuh -- the bookkeeping of a paged key/value cache:
//   paged_plan_kernel    pages, slots and lengths of the next step
//   paged_append_kernel  new K and V rows into the pool
#pragma once

#include "paged_index.h"
#include "paged_ptx.cuh"

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
// entry popped was there before the call.
//
// A latency problem: two block scans over the requests, then independent
// copies of pages and stores of slots, which find their request by bisection
// in shared memory.  One cluster of 16 blocks, each with the whole scan and a
// share of the stores: the cluster's barrier between the reads and the stores
// lets outputs alias inputs, which a larger grid could not, and for a few
// requests the 16 blocks cost nothing that shows.  Launch included: 8 requests
// 8.4 us; 500 requests, 185,000 slots and 0.4 M pages moved 25 us (311 with one
// block).
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
    int n, max_pages, num_pages, page_size, page_shift, tokens;
};

// Shared memory of a plan over n requests: four int arrays.
__host__ __device__ constexpr size_t plan_smem(int n) { return (size_t)(4 * (n + 1)) * sizeof(int); }

// Exclusive sums of K values over the block; total receives the whole sums.
// Every thread calls it; `scratch` holds K values per warp.
template <int K>
__device__ __forceinline__ void block_exclusive_sums(long long (&v)[K], long long* scratch, long long (&total)[K])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    long long x[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        x[k] = v[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x[k], o);
            if (lane >= o) x[k] += y;
        }
        if (lane == 31) scratch[warp * K + k] = x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        // every warp sums the warps' sums for itself
        const long long mine = lane < warps ? scratch[lane * K + k] : 0;
        long long s = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        total[k] = __shfl_sync(0xffffffffu, s, 31);
        v[k] = x[k] - v[k] + __shfl_sync(0xffffffffu, s - mine, warp);
    }
    __syncthreads();     // scratch may be used again
}

__device__ __forceinline__ long long block_exclusive_sum(long long v, long long* scratch, long long* total)
{
    long long x[1] = {v}, t[1];
    block_exclusive_sums<1>(x, scratch, t);
    *total = t[0];
    return x[0];
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

constexpr int kPlanCluster = 16;

// Barrier of all threads of the cluster, with what they wrote before it.
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PlanParams p)
{
    extern __shared__ int plan_smem_raw[];
    __shared__ long long scratch[64];
    __shared__ unsigned long long s_taken;
    __shared__ int s_refused;
    int* s_cu = plan_smem_raw;              // [n + 1] exclusive sums of the new tokens
    int* s_take = s_cu + (p.n + 1);         // [n + 1] exclusive sums of the granted pages
    int* s_rel = s_take + (p.n + 1);        // [n + 1] exclusive sums of the released pages
    int* s_len = s_rel + (p.n + 1);         // [n] cached tokens, or ~tokens if not granted
    const int tid = threadIdx.x, n = p.n, ps = p.page_size;
    const int thread = blockIdx.x * kPlanThreads + tid, threads = gridDim.x * kPlanThreads;
    const int capacity = p.max_pages * ps;  // at most 2^30
    const int per = (n + kPlanThreads - 1) / kPlanThreads;
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    auto page_of = [&](int x) { return page_index(x, ps, p.page_shift); };
    auto pages = [&](int x) { return page_of(x + ps - 1); };
    auto length = [&](int i) { return min(max(p.seq_lens[i], 0), capacity); };
    if (tid == 0) {
        s_taken = ~0ull;
        s_refused = 0;
    }

    const int F = min(max(p.counts[0], 0), p.num_pages);
    long long sums[2] = {0, 0}, totals[2], need_total;      // new tokens, released pages
    for (int i = i0; i < i1; ++i) {
        const int q = p.new_lens[i], have = pages(length(i));
        sums[0] += max(q, 0);
        sums[1] += q < 0 ? have : 0;
    }
    block_exclusive_sums<2>(sums, scratch, totals);
    const long long add0 = sums[0], rel0 = sums[1], add_total = totals[0], rel_total = totals[1];
    const long long A = F + rel_total;
    // pages the request would need: 0 if it does not fit its table row or the slots
    auto need_of = [&](int q, int len, long long cu, bool* fits) {
        *fits = q >= 0 && q <= capacity - len && cu + q <= p.tokens;
        return *fits ? pages(len + q) - pages(len) : 0;
    };
    long long need = 0, cu = add0;
    for (int i = i0; i < i1; ++i) {
        bool fits;
        const int q = p.new_lens[i];
        need += need_of(q, length(i), cu, &fits);
        cu += max(q, 0);
    }
    long long before = block_exclusive_sum(need, scratch, &need_total), released = rel0;
    int refused = 0;
    cu = add0;
    for (int i = i0; i < i1; ++i) {
        bool fits;
        const int q = p.new_lens[i], len = length(i);
        const int want = need_of(q, len, cu, &fits);
        const bool granted = fits && (want == 0 || before + want <= A);
        s_cu[i] = (int)min(cu, (long long)INT_MAX);
        s_take[i] = (int)min(before, A);     // requests past A get nothing
        s_rel[i] = (int)released;
        s_len[i] = granted ? len : ~len;
        refused += q >= 0 && !granted;
        // pages handed out are those before the first request that goes without
        if (fits && !granted) atomicMin(&s_taken, (unsigned long long)before);
        before += want;
        cu += max(q, 0);
        if (q < 0) released += pages(len);
    }
    if (refused) atomicAdd(&s_refused, refused);
    if (tid == 0) {
        s_cu[n] = (int)min(add_total, (long long)INT_MAX);
        s_take[n] = (int)min(need_total, A);
        s_rel[n] = (int)rel_total;
    }
    __syncthreads();
    // every block of the cluster has read every input length and count
    cluster_barrier();
    const int taken = (int)min((long long)min(s_taken, (unsigned long long)need_total), A);

    // A page of the stack, as it stands after the releases.
    auto stack = [&](int x) {
        if (x < F) return p.free_list[x];
        const int j = find_last_le(s_rel, n, x - F);
        return p.table[j * p.table_stride + (x - F - s_rel[j])];
    };
    // to(request, index) = from(request, index) for the indexes below total of
    // the list whose requests begin at start[0 .. n].  A warp takes as many
    // neighbours as give every warp some, 32 at a time, four reads of a lane in
    // flight: a lane bisects for its first index only and then walks on.
    auto for_each = [&](const int* start, int total, auto from, auto to) {
        const int groups = (total + threads - 1) / threads;      // of 32 indexes to a warp
        const long long base = (long long)(thread >> 5) * groups * 32 + (tid & 31);
        if (base >= total) return;
        int i = find_last_le(start, n, (int)base);
        for (int k0 = 0; k0 < groups; k0 += 4) {
            int x[4], at[4], value[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = (int)min(base + 32ll * (k0 + e), (long long)total - 1);
                if (x[e] >= start[i + 1]) {
                    ++i;
                    if (x[e] >= start[i + 1]) i = find_last_le(start, n, x[e]);
                }
                at[e] = i;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) value[e] = from(at[e], x[e]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (k0 + e < groups && base + 32ll * (k0 + e) < total) *to(at[e], x[e]) = value[e];
        }
    };
    if (blockIdx.x == 0) {
        for (int i = tid; i < n; i += kPlanThreads) {
            const int q = p.new_lens[i], l = s_len[i];
            const int len = l < 0 ? ~l : l;
            p.seq_out[i] = q < 0 ? 0 : (l < 0 ? len : len + q);
            p.cu_q[i] = s_cu[i];
        }
        if (tid == 0) {
            p.cu_q[n] = s_cu[n];
            p.counts_out[0] = (int)min(A - taken, (long long)p.num_pages);
            p.counts_out[1] = s_refused;
        }
    }
    for_each(
        s_rel, (int)min(rel_total, (long long)p.num_pages - F),
        [&](int j, int k) { return p.table[j * p.table_stride + (k - s_rel[j])]; },
        [&](int, int k) { return p.free_list + F + k; });
    for_each(
        s_take, taken, [&](int, int k) { return stack((int)A - 1 - k); },
        [&](int i, int k) { return p.table + i * p.table_stride + pages(s_len[i]) + (k - s_take[i]); });
    // the table is complete for every block of the cluster
    cluster_barrier();
    const int named = min(p.tokens, s_cu[n]);
    for_each(
        s_cu, named,
        [&](int i, int t) {
            const int len = s_len[i], pos = max(len, 0) + (t - s_cu[i]);
            const int index = page_of(min(pos, capacity - 1));
            const int page = __ldcg(p.table + i * p.table_stride + index);
            return len >= 0 && page_ok(page, p.num_pages) ? page * ps + (pos - index * ps) : -1;
        },
        [&](int, int t) { return p.slots + t; });
    for (int t = named + thread; t < p.tokens; t += threads) p.slots[t] = -1;
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
