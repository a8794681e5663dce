// draft_verify.cuh -- verification of drafted tokens against the target's
// probabilities, with given random numbers.
//
// Rows cu[i] .. cu[i + 1] - 1 of request i hold the tokens of a step: the last
// one that stands, then those drafted.  Row r of the target is its
// distribution behind token r, row r of the draft's what token r was drawn
// from.  Token r stands if those before it do and
//     u_r draft[r, id_r] < target[r - 1, id_r].
// The token behind the last one that stands is drawn from w = max(target -
// draft, 0) of the first one that does not, or, where all stand, from the
// target's last row: the smallest x with w_0 + .. + w_x > v sum w.
#pragma once

#include "paged_cache.cuh"

namespace ra {
namespace draft {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxVocab = 1 << 18;

struct Params {
    const float* target;
    long long target_stride;
    const float* draft;      // null: the drafted token itself, with probability 1
    long long draft_stride;
    const int* ids;
    const float* u;
    const float* v;
    const int* cu_q;
    int n, tokens, vocab, cluster;
    int* accepted;
    int* next_ids;
    int* drop;
};

// A probability in units of 2^-44, cut to whole ones: 2^22 upper + lower, each
// part kOffset too large.  What is no number or below 0 is 0, what is above 1
// is 1.  Sums of up to 2^18 of them are exact in 64 bits, so they do not depend
// on how the row is shared out, and the token drawn is the same in any order.
// What is cut off counts against the sum that is drawn from: where that is below
// kLeast units the weights are taken again in finer ones (see draw).
//
// An addition of 2, rounded down, leaves 22 bits behind the point in a float's
// last bits.  (Conversions to 64-bit integers run at one or two a cycle and SM:
// with them 64 requests over 131071 tokens took 46 us instead of 20.)
struct Fixed {
    int upper, lower;
    static constexpr int kOffset = 0x40000000;     // 2.f
    __device__ __forceinline__ explicit Fixed(float x)
    {
        x = __saturatef(x);
        const float y = __fadd_rz(x, 2.f);
        upper = __float_as_int(y);
        lower = __float_as_int(__fmaf_rz(x - (y - 2.f), 4194304.f, 2.f));
    }
    __device__ __forceinline__ unsigned long long value() const
    {
        return (unsigned long long)(((long long)(upper - kOffset) << 22) + (lower - kOffset));
    }
};

// max(a - b, 0)
__device__ __forceinline__ unsigned long long above(const Fixed& a, const Fixed& b)
{
    const long long x = ((long long)(a.upper - b.upper) << 22) + (a.lower - b.lower);
    return x > 0 ? (unsigned long long)x : 0ull;
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ unsigned long long warp_inclusive_sum(unsigned long long x)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// What the token behind is drawn from.
enum class Weights { kTarget, kRest, kOthers };     // a row, max(target - draft, 0), a row without one token

// A weight in units of 2^-44, or, kFiner, of 2^-44 / scale, from a target's and a
// draft's probability.  kFiner, a difference is taken in fp32 first, off by 2^-24 of
// itself, and is 0 only where it is none; a power of two as scale rounds nothing.
template <Weights kWhat, bool kFiner>
__device__ __forceinline__ unsigned long long weight(float target, float draft, float scale)
{
    if constexpr (kFiner) {
        float w = __saturatef(target);
        if constexpr (kWhat == Weights::kRest) w = w - __saturatef(draft);
        return Fixed(w * scale).value();
    } else if constexpr (kWhat == Weights::kRest) {
        return above(Fixed(target), Fixed(draft));
    } else {
        return Fixed(target).value();
    }
}

// A row's weights: of a request's target and, for kRest, its draft; kOthers,
// token `gone` has none.
template <Weights kWhat, bool kFiner>
struct Row {
    const float* target;
    const float* draft;
    int gone;
    float scale;
    __device__ __forceinline__ unsigned long long at(int x) const
    {
        if (kWhat == Weights::kOthers && x == gone) return 0ull;
        return weight<kWhat, kFiner>(target[x], kWhat == Weights::kRest ? draft[x] : 0.f, scale);
    }
    // Sum of the weights of tokens x, x + step, ... below x1, kAhead of them loaded
    // in front of their sums: all at once from one row; from two, whose values would
    // take all of the 32 registers, the compiler holds fewer.  (64 requests over
    // 131071 tokens, two rows, 18.4 us, 18.8 with 8; 40 registers and six blocks to
    // an SM, 22.2.)
    __device__ __forceinline__ unsigned long long sum(int x, int x1, int step) const
    {
        constexpr int kAhead = kFiner ? 4 : 16;
        unsigned long long sum = 0;
        for (; x + (kAhead - 1) * step < x1; x += kAhead * step) {
            float f[kAhead], g[kAhead];
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                f[e] = target[x + e * step];
                g[e] = 0.f;
                if constexpr (kWhat == Weights::kRest) g[e] = draft[x + e * step];
            }
#pragma unroll
            for (int e = 0; e < kAhead; ++e)
                if (!(kWhat == Weights::kOthers && x + e * step == gone))
                    sum += weight<kWhat, kFiner>(f[e], g[e], scale);
        }
        for (; x < x1; x += step) sum += at(x);
        return sum;
    }
};

struct Shared {
    unsigned long long warp[kWarps];   // sums of the warps' stretches
    unsigned long long block[2];       // the block's sum, read by the cluster; of two tries in turn
    int accepted;
};

// The least sum that a token is drawn from: up to 2^18 weights, cut by a unit at
// most, then lose 2^-18 of it at most, and half of that on average.
constexpr unsigned long long kLeast = 1ull << 36;
// log2 of the finest scale: units of 2^-149, of which every float is a whole number.
constexpr int kFinest = 105;

// Sums a row's weights and draws a token from them, if the sum is enough or the
// unit the finest; returns the sum.  `turn` counts the calls.
template <Weights kWhat, bool kFiner>
__device__ __forceinline__ unsigned long long try_draw(const Params& p, const Row<kWhat, kFiner>& row, bool finest,
                                                       float v, int rank, int turn, Shared& s, int* next_id)
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int each = ((p.vocab + p.cluster * kWarps - 1) / (p.cluster * kWarps) + 31) / 32 * 32;
    const int x0 = min(p.vocab, (rank * kWarps + warp) * each), x1 = min(p.vocab, x0 + each);
    const unsigned long long mine = warp_sum(row.sum(x0 + lane, x1, 32));
    // (the sums of the try before were read in front of the cluster's barrier there)
    if (lane == 0) s.warp[warp] = mine;
    __syncthreads();
    // every warp knows the sums of those in front of it
    const unsigned long long upto = warp_inclusive_sum(lane < kWarps ? s.warp[lane] : 0ull);
    const unsigned long long block = __shfl_sync(0xffffffffu, upto, 31);
    unsigned long long* given = &s.block[turn & 1];
    if (threadIdx.x == 0) *given = block;
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    unsigned long long other = 0;
    if (lane < p.cluster) {
        uint32_t at;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(given)), "r"(lane));
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(other) : "r"(at) : "memory");
    }
    const unsigned long long blocks = warp_inclusive_sum(other);
    const unsigned long long sum = __shfl_sync(0xffffffffu, blocks, 31);
    if (sum == 0 || (sum < kLeast && !finest)) return sum;
    // v in units of 2^-64, below 1
    const float below = fminf(v, 0.99999994f) * 18446744073709551616.f;
    const unsigned long long share = v > 0.f ? (unsigned long long)below : 0ull;
    const unsigned long long limit = __umul64hi(sum, share);      // floor(v sum), below sum
    unsigned long long at = __shfl_sync(0xffffffffu, blocks - other, rank) +
                            __shfl_sync(0xffffffffu, upto, warp) - mine;
    if (limit < at || limit - at >= mine) return sum;
    // this warp's stretch holds it: a lane sums a piece of neighbours, then the
    // warp scans the piece that holds it
    const int piece = each / 32, p0 = min(x1, x0 + lane * piece), p1 = min(x1, p0 + piece);
    const unsigned long long own = row.sum(p0, p1, 1);
    at += warp_inclusive_sum(own) - own;
    const int holder = __ffs(__ballot_sync(0xffffffffu, limit >= at && limit - at < own)) - 1;
    at = __shfl_sync(0xffffffffu, at, holder);
    const int y1 = __shfl_sync(0xffffffffu, p1, holder);
    for (int y = __shfl_sync(0xffffffffu, p0, holder); y < y1; y += 32) {
        const unsigned long long w = y + lane < y1 ? row.at(y + lane) : 0ull;
        const unsigned long long sums = at + warp_inclusive_sum(w);
        const unsigned found = __ballot_sync(0xffffffffu, limit < sums);
        if (found) {
            if (lane == 0) *next_id = y + __ffs(found) - 1;
            break;
        }
        at = __shfl_sync(0xffffffffu, sums, 31);
    }
    return sum;
}

// The tries behind a first one whose sum was not enough; false if all weights are 0.
// (A function of its own, as it is rare: inside the kernel its registers would
// be spilled by the first try.)
template <Weights kWhat>
__device__ __noinline__ bool draw_finer(const Params& p, const float* target, const float* draft, int gone, float v,
                                        int rank, int turn, Shared& s, int* next_id, unsigned long long sum)
{
    for (int finer = 0; sum < kLeast && finer < kFinest;) {
        finer = min(kFinest, finer + __clzll((long long)sum) - 20);
        sum = try_draw(p, Row<kWhat, true>{target, draft, gone, __int_as_float((127 + finer) << 23)}, finer == kFinest,
                       v, rank, turn++, s, next_id);
    }
    __syncwarp();
    cluster_arrive();      // the blocks' sums have been read, whatever turn comes next
    cluster_wait();
    return sum != 0;
}

// Draws from a row's weights; false if all are 0.  Weights that are small in sum
// (behind a drafted token that held nearly all of the row) are summed again in
// units as fine as the sum allows: none of them is above the sum by a unit, so
// scaled by 2^(44 - bits of the sum) none is above 1, and the sum then has 43 bits
// at least; a sum of 0 says that all are below a unit.  Every block sees the same
// sums.  Two rounds where the first finds something, four at most.
template <Weights kWhat>
__device__ __forceinline__ bool draw(const Params& p, const float* target, const float* draft, int gone, float v,
                                     int rank, int& turn, Shared& s, int* next_id)
{
    const unsigned long long sum =
        try_draw(p, Row<kWhat, false>{target, draft, gone, 1.f}, false, v, rank, turn++, s, next_id);
    return sum >= kLeast || draw_finer<kWhat>(p, target, draft, gone, v, rank, turn, s, next_id, sum);
}

// A cluster to a request; each block sums a stretch of the row, each warp a
// stretch of that, and the warp that holds the token reads its stretch again.
// Bound by HBM for many requests (one row of the target and one of the draft's
// each), by a chain of waits for few: offsets, the token's number, its
// probabilities, the rows, the other blocks' sums, the stretch.  One request over
// 32768 tokens 4.7 us, launch included; 64 over 131071, 17.5 us with the rows in
// L2, 25 us from HBM (0.40 of copy bandwidth: the chain in front of the rows,
// which all blocks wait for at the same time, takes 3 us, what follows as long);
// drafted outright 15.8 and 23; with sums that want a second round 29 and 37.
__global__ void __launch_bounds__(kThreads, 8) draft_verify_kernel(const Params p)
{
    __shared__ Shared s;
    const int i = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
    const int tid = threadIdx.x, lane = tid % 32;
    const int a = min(max(p.cu_q[i], 0), p.tokens), b = min(max(p.cu_q[i + 1], a), p.tokens);
    const float v = p.v[i];
    if (a == b) {      // no token: so for every block of the cluster
        if (rank == 0 && tid == 0) {
            p.accepted[i] = p.drop[i] = 0;
            p.next_ids[i] = -1;
        }
        return;
    }
    if (tid < 32) {
        int first = b - a - 1;      // drafted tokens that stand
        for (int r0 = a + 1; r0 < b; r0 += 32) {
            const int r = r0 + lane;
            bool stands = r >= b;
            if (r < b) {
                const int x = p.ids[r];
                const float u = p.u[r];
                if ((unsigned)x < (unsigned)p.vocab) {
                    const double q = p.draft ? p.draft[r * p.draft_stride + x] : 1.f;
                    stands = u * q < p.target[(r - 1) * p.target_stride + x];   // the product is exact
                }
            }
            const unsigned refused = __ballot_sync(0xffffffffu, !stands);
            if (refused) {
                first = r0 - a - 1 + __ffs(refused) - 1;
                break;
            }
        }
        if (lane == 0) s.accepted = first;
    }
    __syncthreads();
    const int accepted = s.accepted, row = a + accepted;
    const float* target = p.target + row * p.target_stride;
    bool drawn = false;
    int turn = 0;
    if (row + 1 < b) {
        // the first token that does not stand
        if (p.draft)
            drawn = draw<Weights::kRest>(p, target, p.draft + (row + 1) * p.draft_stride, -1, v, rank, turn, s,
                                         p.next_ids + i);
        else drawn = draw<Weights::kOthers>(p, target, nullptr, p.ids[row + 1], v, rank, turn, s, p.next_ids + i);
    }
    // all stand, or nothing is left: the target's row itself
    if (!drawn) drawn = draw<Weights::kTarget>(p, target, nullptr, -1, v, rank, turn, s, p.next_ids + i);
    if (rank == 0 && tid == 0) {
        p.accepted[i] = accepted;
        p.drop[i] = b - a - 1 - accepted;
        if (!drawn) p.next_ids[i] = -1;
    }
    // a block stays until no other reads its sums
    __syncwarp();
    cluster_arrive();
    cluster_wait();
}

}  // namespace draft
}  // namespace ra
