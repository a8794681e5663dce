// rope.cuh -- norm and rotation of queries and keys:
//   rope_fwd_kernel          q and k, or a step's tokens into a paged cache; without
//                            norms the backward pass too, which turns back
//   rope_bwd_kernel          gradients of the rows and parts of the weights'
//   rope_weight_grad_kernel  the weights' gradients from those parts
//
// A row x of d elements becomes
//     x' = x w / sqrt(mean x^2 + eps)        (where there are weights)
//     y_a = x'_a c_i - x'_b s_i,  y_b = x'_b c_i + x'_a s_i
// for the pairs (a, b) of the first `rot` elements, c_i and s_i the cosine and
// the sine of position * inv_freq[i] times the amplitude; pair i is (i, i + rot
// / 2) in the half layout, (2 i, 2 i + 1) in the interleaved one.  Backwards,
// with r = 1 / sqrt(mean x^2 + eps) and g' the gradient turned back:
//     g = g' w,  dx = r (g - x r^2 mean(g x)),  dw = sum over rows g' x r.
//
// Bound by HBM: 4 bytes an element forwards, 6 backwards (4 without norms).
// A lane holds 16 elements of a row, chosen so that pairs never cross lanes: no
// exchange but the norm's sums, and what a row costs beside its elements
// (addresses, sums over the lanes, the root) is shared by twice as many as with 8.
// Measured at the 128K grouped-query shape (32 heads over 8, d 128, bf16, parts
// of one projection's rows): forwards 402 us, 1.00 of measured copy bandwidth;
// backwards 649 us, 0.93, an instruction in half of the cycles.
#pragma once

#include "paged_attn.cuh"

namespace ra {
namespace rope {

constexpr int kThreads = 128, kWarps = kThreads / 32;
// Blocks to an SM and rows of a batch (kUnroll, kBackUnroll): registers spent on
// rows in flight, in stretches of memory as long as can be, count for more than
// warps.  128K grouped-query shape: forwards 3 rows to a lane group with 16 warps
// to an SM 402 us, 2 rows 413, 4 rows with 12 warps 423, 1 row with 24 warps 474;
// backwards 2 rows with 12 warps 648, with 16 (spilled) 932, 1 row with 16 825.
constexpr int kBlocksPerSm = 4, kBackPerSm = 3;
constexpr int kMaxBlocks = 160 * kBackPerSm;      // whose sums are kept

// Rows of one tensor: (batch, position, head) to element offsets, and where
// their results go.
struct Rows {
    const uint16_t* x;      // input; null in a backward pass without norm
    long long xb, xs, xh;
    const uint16_t* g;      // backward: gradient of the output
    long long gb, gs, gh;
    uint16_t* out;
    long long ob, os, oh;
    const float* w;         // null: no norm
    int heads;
};

struct Params {
    Rows q, k;
    const int* positions;
    long long pos_batch;    // 0: the same positions in every batch row
    const float* inv_freq;
    float eps, amplitude, sign;   // sign -1 turns back
    int rot, interleaved, S, tokens, parts;
    float* partial;         // backward: [blocks][2][d] sums of the weights' gradients
};

// A step's tokens into a paged cache.
struct Paged {
    const uint16_t* v;
    long long vs, vh;
    uint16_t* kc;
    paged::PoolLayout lk;
    uint16_t* vc;
    paged::PoolLayout lv;
    const int* slots;
    const int* seq_lens;
    const int* cu_q;
    int n, page_size, num_slots;
    uint32_t* status;
};

// f / (2 pi) modulo 1, in units of 2^-64 of a turn: a position's angle is then
// a product modulo 2^64, exact to 2^-64 of a turn for each position, however
// far.  f = m 2^-s, below 2^26, is multiplied by 2^130 / (2 pi) in two words: with
// one, 2^66 / (2 pi), frequencies from 2^8 on would be off by more than a unit,
// those near 2^26 by 2^18 of them.
__device__ __forceinline__ uint64_t turn_of(float f)
{
    constexpr uint64_t kTurn = 0xa2f9836e4e441529ull, kRest = 0xfc2757d1f534ddc0ull;
    const uint32_t bits = __float_as_uint(f);
    const uint32_t e = max(bits >> 23 & 255u, 1u);
    const uint64_t m = (bits & 0x7fffffu) | (bits & 0x7f800000u ? 0x800000u : 0u);
    const uint64_t carried = __umul64hi(m, kRest), lo = m * kTurn + carried;
    const uint64_t hi = __umul64hi(m, kTurn) + (lo < carried);
    const int shift = 152 - (int)e;
    uint64_t t = 0;
    if (shift >= 64) t = shift < 128 ? hi >> (shift - 64) : 0ull;
    else if (shift > 0) t = lo >> shift | hi << (64 - shift);
    else if (shift > -64) t = lo << -shift;
    return bits >> 31 ? 0ull - t : t;
}

// How the lanes of a warp share rows of D elements: lane l of a group of kLanes
// holds the octets (8 elements) first and second of the group's row.  Lanes
// below rot / 16 hold pairs 8 l .. 8 l + 7, the others what is not rotated.
template <int D>
struct Place {
    static constexpr int kLanes = D / 16, kGroups = 32 / kLanes;
    int l, group, first, second;
    bool turns;
    __device__ __forceinline__ Place(int rot, bool interleaved)
    {
        const int lane = threadIdx.x & 31;
        l = lane % kLanes;
        group = lane / kLanes;
        turns = l < rot / 16;
        first = turns && !interleaved ? 8 * l : 16 * l;
        second = turns && !interleaved ? first + rot / 2 : first + 8;
    }
};

// Cosines and sines of a warp's token, in shared memory: every lane computes
// its share of the D / 2 pairs.
template <int D>
struct Angles {
    static constexpr int kEach = D / 64;
    uint64_t turn[kEach];
    float* c;      // [D / 2], then the sines
    __device__ __forceinline__ Angles(const Params& p, float* shared) : c(shared)
    {
        const int pair = (threadIdx.x & 31) * kEach;
#pragma unroll
        for (int i = 0; i < kEach; ++i) turn[i] = pair + i < p.rot / 2 ? turn_of(p.inv_freq[pair + i]) : 0ull;
    }
    __device__ __forceinline__ void at(int position, float amplitude, float sign) const
    {
        const int pair = (threadIdx.x & 31) * kEach;
        float cs[kEach], sn[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const long long angle = (long long)(turn[i] * (uint64_t)(long long)position);
            sincospif((float)angle * 1.0842021724855044e-19f, &sn[i], &cs[i]);      // 2^-63
            cs[i] *= amplitude;
            sn[i] *= sign * amplitude;
        }
        __syncwarp();       // the token before this one has been turned
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            c[pair + i] = cs[i];
            c[D / 2 + pair + i] = sn[i];
        }
        __syncwarp();
    }
};

// Two floats in one register pair, for the packed instructions.
struct F2 {
    uint64_t x;
};
__device__ __forceinline__ F2 make_f2(float lo, float hi)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.x) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split(F2 v, float& lo, float& hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v.x));
}
__device__ __forceinline__ F2 mul(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.x) : "l"(a.x), "l"(b.x));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.x) : "l"(a.x), "l"(b.x), "l"(c.x));
    return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.x) : "l"(a.x), "l"(b.x));
    return r;
}
__device__ __forceinline__ float sum_of(F2 v)
{
    float lo, hi;
    split(v, lo, hi);
    return lo + hi;
}

template <bool kHalf>
__device__ __forceinline__ F2 widen2(uint32_t x)
{
    if constexpr (kHalf) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
        return make_f2(f.x, f.y);
    } else {
        return make_f2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    }
}

// The lane's elements of a row, so that rotation pairs are v[j] and v[4 + j]: its
// first octet, then the second; interleaved, the even elements of its sixteen
// neighbours, then the odd ones.
using Sixteen = F2[8];

// Four pairs from shared memory.
__device__ __forceinline__ void load_pairs(F2* to, const float* from)
{
    const float4 a = *reinterpret_cast<const float4*>(from), b = *reinterpret_cast<const float4*>(from + 4);
    to[0] = make_f2(a.x, a.y);
    to[1] = make_f2(a.z, a.w);
    to[2] = make_f2(b.x, b.y);
    to[3] = make_f2(b.z, b.w);
}

// Sixteen neighbours to even and odd ones.
__device__ __forceinline__ void part(Sixteen& v)
{
    float x[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) split(v[j], x[2 * j], x[2 * j + 1]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = make_f2(x[4 * j], x[4 * j + 2]);
        v[4 + j] = make_f2(x[4 * j + 1], x[4 * j + 3]);
    }
}

// Two octets of a row as they lie in memory.
struct Octets {
    uint4 a, b;
    template <int D> __device__ __forceinline__ void load(const uint16_t* row, const Place<D>& at)
    {
        a = *reinterpret_cast<const uint4*>(row + at.first);
        b = *reinterpret_cast<const uint4*>(row + at.second);
    }
    template <int D> __device__ __forceinline__ void store(uint16_t* row, const Place<D>& at) const
    {
        *reinterpret_cast<uint4*>(row + at.first) = a;
        *reinterpret_cast<uint4*>(row + at.second) = b;
    }
    template <bool kHalf, bool kInter> __device__ __forceinline__ void widen(Sixteen& v) const
    {
        const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = widen2<kHalf>(x[j]);
        if constexpr (kInter) part(v);
    }
    // The one rounding of a row.
    template <bool kHalf, bool kInter> __device__ __forceinline__ void pack(const Sixteen& v)
    {
        uint32_t out[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float lo, hi;
            if constexpr (kInter) {
                float x[2], y[2];
                split(v[j / 2], x[0], x[1]);
                split(v[4 + j / 2], y[0], y[1]);
                lo = x[j & 1];
                hi = y[j & 1];
            } else {
                split(v[j], lo, hi);
            }
            out[j] = paged::Operand<kHalf>::pack(lo, hi);
        }
        a = make_uint4(out[0], out[1], out[2], out[3]);
        b = make_uint4(out[4], out[5], out[6], out[7]);
    }
};

// kCount rows of a tensor, one to a lane group and step: heads h, h + kGroups, ...
template <int D, int kCount>
struct Batch {
    Octets row[kCount];
    __device__ __forceinline__ void load(const uint16_t* x, long long xh, int h, int hi, const Place<D>& at)
    {
        const uint16_t* from = x + h * xh;
#pragma unroll
        for (int e = 0; e < kCount; ++e) {
            row[e].a = row[e].b = make_uint4(0u, 0u, 0u, 0u);
            if (h + e * Place<D>::kGroups < hi) row[e].load(from, at);
            from += Place<D>::kGroups * xh;
        }
    }
};

// The lane's weights, in the order of its elements.
template <int D, bool kInter>
__device__ __forceinline__ void load_weights(Sixteen& w, const float* from, const Place<D>& at)
{
    load_pairs(w, from + at.first);
    load_pairs(w + 4, from + at.second);
    if constexpr (kInter) part(w);
}

// The turn of the lane's elements with the weights of a norm in it, y = v *
// same + partner(v) * other.  What is not turned is not even multiplied by 0: it
// may be infinite.
template <int D, bool kInter>
struct WeightedTurn {
    Sixteen same, other;
    __device__ __forceinline__ WeightedTurn(const float* cs, const float* weights, const Place<D>& at)
    {
        Sixteen w;
        load_weights<D, kInter>(w, weights, at);
        F2 c[4], s[4];
        const int pair = at.turns ? 8 * at.l : 0;
        load_pairs(c, cs + pair);
        load_pairs(s, cs + D / 2 + pair);
        const F2 minus = make_f2(-1.f, -1.f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            same[j] = at.turns ? mul(c[j & 3], w[j]) : w[j];
            other[j] = mul(j < 4 ? mul(s[j & 3], minus) : s[j & 3], w[j ^ 4]);
        }
    }
    __device__ __forceinline__ void operator()(Sixteen& y, const Sixteen& v, bool turns) const
    {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = mul(v[j], same[j]);
        if (turns) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = fma(v[j ^ 4], other[j], y[j]);
        }
    }
};

// The turn alone, with fewer registers.
template <int D>
struct Turn {
    F2 c[4], s[4];
    __device__ __forceinline__ Turn(const float* cs, const Place<D>& at)
    {
        const int pair = at.turns ? 8 * at.l : 0;
        load_pairs(c, cs + pair);
        load_pairs(s, cs + D / 2 + pair);
    }
    __device__ __forceinline__ void operator()(Sixteen& v, bool turns) const
    {
        if (!turns) return;
        const F2 minus = make_f2(-1.f, -1.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const F2 a = v[j], b = v[4 + j];
            v[j] = fma(mul(b, minus), s[j], mul(a, c[j]));
            v[4 + j] = fma(a, s[j], mul(b, c[j]));
        }
    }
};

template <int kLanes>
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Both tensors' weights into shared memory, [2][D], 1 without a norm.
template <int D>
__device__ __forceinline__ void share_weights(float* to, const Params& p)
{
    for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
        const float* w = x < D ? p.q.w : p.k.w;
        to[x] = w ? w[x % D] : 1.f;
    }
    __syncthreads();
}

// A warp's place in the list of (token, share of its heads).
struct Item {
    int t, lo, hi, b, pos;
    __device__ __forceinline__ Item(const Params& p, unsigned item, int all, int share, bool batches)
    {
        t = (int)item;
        lo = 0;
        if (p.parts > 1) {
            t = (int)(item / (unsigned)p.parts);
            lo = (int)(item % (unsigned)p.parts) * share;
        }
        hi = min(all, lo + share);
        b = batches && p.S < p.tokens ? t / p.S : 0;
        pos = t - b * p.S;
    }
};

// Last request whose tokens begin at or before t, -1 if t is no request's.
// The warp looks at 32 of them at a time.
__device__ __forceinline__ int request_of(const int* cu_q, int n, int t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n;
    while (len > 1) {
        const int step = (len + 31) / 32, i = lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, i < len && cu_q[lo + min(i, len - 1)] <= t);
        const int skip = max(__popc(below) - 1, 0) * step;      // below len, as only lanes below it vote
        lo += skip;
        len = min(step, len - skip);
    }
    return cu_q[lo] <= t && t < cu_q[lo + 1] ? lo : -1;
}

constexpr int kUnroll = 3;         // rows of a lane group in a batch, forwards
constexpr int kBackUnroll = 2;     // and backwards

// One batch: norm, turn, store.
template <int D, bool kHalf, bool kInter>
__device__ __forceinline__ void turn_batch(Batch<D, kUnroll>& batch, uint16_t* out, long long oh, int h, int hi,
                                           bool norm, float eps, const WeightedTurn<D, kInter>& turn,
                                           const Place<D>& at)
{
    using P = Place<D>;
    uint16_t* to = out + h * oh;
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
        if (e > 0 && h - at.group + e * P::kGroups >= hi) break;      // no row in the warp
        Sixteen v, y;
        batch.row[e].template widen<kHalf, kInter>(v);
        turn(y, v, at.turns);
        if (norm) {
            F2 sum = mul(v[0], v[0]), more = mul(v[1], v[1]);
#pragma unroll
            for (int j = 2; j < 8; j += 2) {
                sum = fma(v[j], v[j], sum);
                more = fma(v[j + 1], v[j + 1], more);
            }
            const float r = rsqrtf(row_sum<P::kLanes>(sum_of(add(sum, more))) * (1.f / D) + eps);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = mul(y[j], make_f2(r, r));
        }
        batch.row[e].template pack<kHalf, kInter>(y);
        if (h + e * P::kGroups < hi) batch.row[e].store(to, at);
        to += P::kGroups * oh;
    }
}

// A warp takes a token, or one of `parts` shares of its heads where there are
// few tokens.  The next batch of rows is on its way while one is turned, the
// first while the angles are computed.  (Shares where tokens alone are enough
// cost: the angles and the set-up are a fifth of a token's instructions, 405 us
// with one and 498 with two.)  Into a paged cache: one token 4.1 us, launch
// included; 4125 tokens of chunks, 32 heads, 38.9 us, 0.88 of copy bandwidth,
// as 1.7 rounds of warps take two.
template <int D, bool kHalf, bool kInter, bool kPaged>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
rope_fwd_kernel(const Params p, const Paged c)
{
    using P = Place<D>;
    constexpr int kStep = P::kGroups * kUnroll;
    __shared__ alignas(16) float s_angles[kWarps][D], s_weights[2 * D];
    const P at(p.rot, kInter);
    const Angles<D> angles(p, s_angles[threadIdx.x / 32]);
    share_weights<D>(s_weights, p);
    const int all = p.q.heads + p.k.heads + (kPaged ? p.k.heads : 0);
    const int share = (all + p.parts - 1) / p.parts;
    const unsigned items = (unsigned)p.tokens * (unsigned)p.parts, warps = gridDim.x * kWarps;    // below 2^31
    for (unsigned item = blockIdx.x * kWarps + threadIdx.x / 32; item < items; item += warps) {
        const Item i(p, item, all, share, !kPaged);
        const int q1 = min(i.hi, p.q.heads), k0 = max(0, i.lo - p.q.heads), k1 = min(i.hi - p.q.heads, p.k.heads);
        const uint16_t* q = p.q.x + i.b * p.q.xb + i.pos * p.q.xs;
        const uint16_t* k = p.k.x + i.b * p.k.xb + i.pos * p.k.xs;
        Batch<D, kUnroll> next;
        if (i.lo < q1) next.load(q, p.q.xh, i.lo + at.group, q1, at);
        else if (k0 < k1) next.load(k, p.k.xh, k0 + at.group, k1, at);
        int position, slot = -1;
        uint16_t *k_out, *v_out = nullptr;
        long long k_out_head;
        if constexpr (kPaged) {
            slot = c.slots[i.t];
            const int r = request_of(c.cu_q, c.n, i.t);
            if (r < 0) continue;
            position = (int)((unsigned)c.seq_lens[r] - (unsigned)c.cu_q[r + 1] + (unsigned)i.t);
        } else {
            position = p.positions[i.b * p.pos_batch + i.pos];
        }
        angles.at(position, p.amplitude, p.sign);
        if (i.lo < q1) {
            const WeightedTurn<D, kInter> turn(angles.c, s_weights, at);
            uint16_t* out = p.q.out + i.b * p.q.ob + i.pos * p.q.os;
            for (int h = i.lo; h < q1; h += kStep) {
                Batch<D, kUnroll> batch = next;
                if (h + kStep < q1) next.load(q, p.q.xh, h + kStep + at.group, q1, at);
                else if (k0 < k1) next.load(k, p.k.xh, k0 + at.group, k1, at);
                turn_batch<D, kHalf, kInter>(batch, out, p.q.oh, h + at.group, q1, p.q.w != nullptr, p.eps, turn, at);
            }
        }
        if constexpr (kPaged) {
            if ((unsigned)slot >= (unsigned)c.num_slots) {
                if (slot != -1 && (threadIdx.x & 31) == 0) atomicOr(c.status, kStatusBadPage);
                continue;
            }
            const int page = slot / c.page_size, off = slot - page * c.page_size;
            k_out = c.kc + row_offset(c.lk, page, off, 0);
            k_out_head = c.lk.sh;
            v_out = c.vc + row_offset(c.lv, page, off, 0);
        } else {
            k_out = p.k.out + i.b * p.k.ob + i.pos * p.k.os;
            k_out_head = p.k.oh;
        }
        if (k0 < k1) {
            const WeightedTurn<D, kInter> turn(angles.c, s_weights + D, at);
            for (int h = k0; h < k1; h += kStep) {
                Batch<D, kUnroll> batch = next;
                if (h + kStep < k1) next.load(k, p.k.xh, h + kStep + at.group, k1, at);
                turn_batch<D, kHalf, kInter>(batch, k_out, k_out_head, h + at.group, k1, p.k.w != nullptr, p.eps, turn,
                                             at);
            }
        }
        if constexpr (kPaged) {
            const int v1 = i.hi - p.q.heads - p.k.heads;
            for (int h = max(0, i.lo - p.q.heads - p.k.heads) + at.group; h - at.group < v1; h += kStep) {
                next.load(c.v + i.t * c.vs, c.vh, h, v1, at);
#pragma unroll
                for (int e = 0; e < kUnroll; ++e)
                    if (h + e * P::kGroups < v1) next.row[e].store(v_out + (h + e * P::kGroups) * c.lv.sh, at);
            }
        }
    }
}

// Gradients of one batch's rows; here: the token's share of the weight's.
template <int D, bool kHalf, bool kInter>
__device__ __forceinline__ void turn_batch_back(Batch<D, kBackUnroll>& g, Batch<D, kBackUnroll>& x, uint16_t* out,
                                                long long oh, int h, int hi, bool norm, float eps, const float* weights,
                                                Sixteen& here, const Turn<D>& turn, const Place<D>& at)
{
    using P = Place<D>;
    uint16_t* to = out + h * oh;
#pragma unroll
    for (int e = 0; e < kBackUnroll; ++e) {
        if (e > 0 && h - at.group + e * P::kGroups >= hi) break;      // no row in the warp
        const bool row = h + e * P::kGroups < hi;
        Sixteen y;
        g.row[e].template widen<kHalf, kInter>(y);
        turn(y, at.turns);
        if (norm) {
            Sixteen v, gw;
            load_weights<D, kInter>(gw, weights, at);
            x.row[e].template widen<kHalf, kInter>(v);
            F2 sum = make_f2(0.f, 0.f), dot = sum;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                gw[j] = mul(gw[j], y[j]);
                sum = fma(v[j], v[j], sum);
                dot = fma(gw[j], v[j], dot);
            }
            const float r = rsqrtf(row_sum<P::kLanes>(sum_of(sum)) * (1.f / D) + eps);
            const float m = -r * r * (row_sum<P::kLanes>(sum_of(dot)) * (1.f / D));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = mul(v[j], make_f2(r, r));
                if (row) here[j] = fma(y[j], v[j], here[j]);
                y[j] = fma(v[j], make_f2(m, m), mul(gw[j], make_f2(r, r)));
            }
        }
        g.row[e].template pack<kHalf, kInter>(y);
        if (row) g.row[e].store(to, at);
        to += P::kGroups * oh;
    }
}

// A warp takes a token, or a share of its heads, as forwards.
template <int D, bool kHalf, bool kInter>
__global__ void __launch_bounds__(kThreads, kBackPerSm) rope_bwd_kernel(const Params p)
{
    using P = Place<D>;
    constexpr int kStep = P::kGroups * kBackUnroll;
    __shared__ alignas(16) float s_angles[kWarps][D], s_weights[2 * D];
    // the weights' gradients, [warp][q, k][quad][lane]: a token's rows are
    // summed first, then tokens here, so that sums stay short
    __shared__ float4 s_sum[kWarps][2][4][32];
    const P at(p.rot, kInter);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const Angles<D> angles(p, s_angles[warp]);
#pragma unroll
    for (int x = 0; x < 8; ++x) s_sum[warp][x / 4][x & 3][lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    share_weights<D>(s_weights, p);
    const int all = p.q.heads + p.k.heads, share = (all + p.parts - 1) / p.parts;
    const unsigned items = (unsigned)p.tokens * (unsigned)p.parts, warps = gridDim.x * kWarps;    // below 2^31
    for (unsigned item = blockIdx.x * kWarps + warp; item < items; item += warps) {
        const Item i(p, item, all, share, true);
        const int position = p.positions[i.b * p.pos_batch + i.pos];
        bool turned = false;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int h0 = x ? max(0, i.lo - p.q.heads) : i.lo;
            const int hi = x ? min(i.hi - p.q.heads, p.k.heads) : min(i.hi, p.q.heads);
            if (h0 >= hi) continue;
            const Rows& r = x ? p.k : p.q;
            const bool norm = r.w != nullptr;
            const uint16_t *from_g = r.g + i.b * r.gb + i.pos * r.gs, *from_x = r.x + i.b * r.xb + i.pos * r.xs;
            Batch<D, kBackUnroll> next_g, next_x;
            next_g.load(from_g, r.gh, h0 + at.group, hi, at);
            if (norm) next_x.load(from_x, r.xh, h0 + at.group, hi, at);
            if (!turned) angles.at(position, p.amplitude, p.sign);
            turned = true;
            const Turn<D> turn(angles.c, at);
            Sixteen here;
#pragma unroll
            for (int j = 0; j < 8; ++j) here[j] = make_f2(0.f, 0.f);
            uint16_t* out = r.out + i.b * r.ob + i.pos * r.os;
            for (int h = h0 + at.group; h - at.group < hi; h += kStep) {
                Batch<D, kBackUnroll> g = next_g, v = next_x;
                next_g.load(from_g, r.gh, h + kStep, hi, at);
                if (norm) next_x.load(from_x, r.xh, h + kStep, hi, at);
                turn_batch_back<D, kHalf, kInter>(g, v, out, r.oh, h, hi, norm, p.eps, s_weights + x * D, here, turn,
                                                  at);
            }
            if (norm) {
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float4 sum = s_sum[warp][x][y][lane];
                    float a[4];
                    split(here[2 * y], a[0], a[1]);
                    split(here[2 * y + 1], a[2], a[3]);
                    s_sum[warp][x][y][lane] = make_float4(sum.x + a[0], sum.y + a[1], sum.z + a[2], sum.w + a[3]);
                }
            }
        }
    }
    if (!p.partial) return;
    // the block's sums, in an order that does not change from call to call
    __syncthreads();
    const float* sums = reinterpret_cast<const float*>(s_sum);
    for (int y = threadIdx.x; y < 2 * D; y += kThreads) {
        const int x = y / D, e = y % D;         // tensor, element: of which lane, and where in its sixteen
        const int half = p.rot / 2, l = e < p.rot && !kInter ? e % half / 8 : e / 16;
        const int in = e < p.rot && !kInter ? e / half * 8 + e % 8 : e % 16;
        const int at = kInter ? in / 4 * 2 + (in & 1) * 8 + (in >> 1 & 1) : in;
        float sum = 0.f;
        for (int w = 0; w < kWarps; ++w)
#pragma unroll
            for (int g = 0; g < P::kGroups; ++g)
                sum += sums[(((w * 2 + x) * 4 + at / 4) * 32 + g * P::kLanes + l) * 4 + at % 4];
        p.partial[(long long)blockIdx.x * 2 * D + y] = sum;
    }
}

// dw of q's weights (blockIdx.y 0) or k's from the blocks' sums: a warp sums a
// column, in a fixed order; 0 from no block.
__global__ void __launch_bounds__(kThreads)
rope_weight_grad_kernel(const float* __restrict__ partial, int blocks, int d, float* dwq, float* dwk)
{
    paged::wait_for_previous();
    float* out = blockIdx.y ? dwk : dwq;
    const int col = blockIdx.x * kWarps + threadIdx.x / 32, lane = threadIdx.x & 31;
    if (!out || col >= d) return;
    float sum = 0.f;
    #pragma unroll 4
    for (int b = lane; b < blocks; b += 32) sum += partial[((long long)b * 2 + blockIdx.y) * d + col];
    sum = row_sum<32>(sum);
    if (lane == 0) out[col] = sum;
}

}  // namespace rope
}  // namespace ra
