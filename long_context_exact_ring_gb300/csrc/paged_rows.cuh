// paged_rows.cuh -- attention of few new tokens over a paged cache: the form
// of paged_attn_fwd for decode steps.
#pragma once

#include "paged_attn.cuh"

namespace ra {
namespace paged {
namespace rows {

constexpr int kRows = kRowsTile;        // packed rows of a tile: one m16n8k16 operand
constexpr int kWarps = 8;               // that compute
constexpr int kThreads = 384;
// Warp 0 copies, warps 4-11 compute; 1-3 lend them their registers: 128 * 72 +
// 256 * 216 are the 384 * 168 that the block starts with.
constexpr int kFewRegs = 72, kManyRegs = 216;

template <int D>
struct Cfg {
    // Keys of a warp's step, and of the block's, the smallest piece of work: a
    // step is a chain of waits, products and shuffles, so with half the bytes
    // to a key it takes twice the keys.
    static constexpr int kKeys = D == 128 ? 16 : 32;
    static constexpr int kUnit = kKeys * kWarps;
    static constexpr int kBoxes = D / 64;                          // 64-column boxes of a row
    static constexpr int kBoxBytes = 64 * kUnit * 2;
    static constexpr int kTileBytes = kUnit * D * 2;               // K (or V) of a unit
    static constexpr int kStages = 3;
    static constexpr int kOffSums = 2 * kStages * kTileBytes;      // [warp][8 rows][D] of half a tile
    static constexpr int kOffStat = kOffSums + kWarps * 8 * D * 4; // [2][warp][8 rows] references, sums
    static constexpr int kOffBar = kOffStat + 2 * kWarps * 8 * 4;
    static constexpr int kSmemBytes = kOffBar + 256 + 1024;        // + alignment slack
};

// What a tile costs beside its keys, in units: the states of eight warps are
// merged and the results written, 2 to 3 us against 1.5 us for a unit.  64
// ragged contexts up to 16K, on one box in turn: 342 us without it, 333 with 1,
// 329 with 2; 64 contexts of up to 1153 keys, 32 heads of 64: 120, 88 and 76 us.
constexpr int kExtra = 2;

constexpr float kLeastBf16 = 9.18354962e-41f;    // 2^-133

// A block's place in its share: units [u0, u1) of kUnit keys of a tile.
template <int kUnit>
struct Walk {
    const AttnParams& p;
    const RowRange& range;
    Request r;
    int req, item, tiles, units, u0, u1;    // item: key/value head x tile of the request
    long long left;                         // cost of what follows this piece

    static __device__ __forceinline__ int tiles_of(const AttnParams& p, const Request& r)
    {
        return (r.q * p.group + kRows - 1) / kRows;
    }
    static __device__ __forceinline__ int units_of(const Request& r) { return max(1, (r.len + kUnit - 1) / kUnit); }
    static __device__ __forceinline__ long long cost(const AttnParams& p, const RowRange& range, int i)
    {
        const Request r = load_request(p, i);
        return range.has(r.q * p.group) ? (long long)tiles_of(p, r) * p.kv_heads * (units_of(r) + kExtra) : 0ll;
    }
    __device__ __forceinline__ Walk(const AttnParams& p_, const RowRange& range_, int req_, long long offset,
                                    long long share)
        : p(p_), range(range_), req(req_), left(share)
    {
        load();
        item = quotient_below(offset, units + kExtra, tiles * p.kv_heads);
        cut(offset - (long long)item * (units + kExtra));
    }
    __device__ __forceinline__ void load()
    {
        r = load_request(p, req);
        tiles = tiles_of(p, r);
        units = units_of(r);
    }
    // The piece that begins at cost c0 of the tile.
    __device__ __forceinline__ void cut(long long c0)
    {
        const long long c1 = min((long long)units + kExtra, c0 + left);
        left -= c1 - c0;
        u0 = cut_units(c0, kExtra);
        u1 = cut_units(c1, kExtra);
    }
    // The share ends in front of the tile's first key.
    __device__ __forceinline__ bool empty() const { return u0 == u1; }
    __device__ __forceinline__ int kvh() const { return tiles == 1 ? item : item / tiles; }
    __device__ __forceinline__ int row0() const { return tiles == 1 ? 0 : item % tiles * kRows; }
    __device__ __forceinline__ int rows() const { return min(kRows, r.q * p.group - row0()); }
    // behind the last key of this piece that a row of the tile sees
    __device__ __forceinline__ int keys() const
    {
        const int last = (row0() + rows() - 1) / p.group;      // last token
        return min(u1 * kUnit, p.causal ? r.len - r.q + last + 1 : r.len);
    }
    // To the next piece of work; false behind the last one.
    __device__ __forceinline__ bool next()
    {
        if (left == 0) return false;
        if (++item == tiles * p.kv_heads) {
            item = 0;
            do {
                ++req;
                load();
            } while (!range.has(r.q * p.group));     // some later request has the work that is left
        }
        cut(0);
        return !empty();
    }
};

struct RowsParams {
    AttnParams a;
    Workspace ws;
    RowRange range;
    int box_rows;            // rows of a K/V box: the largest power of two in page_size, at most 128
    uint64_t wait_limit_ns;
};

// The work is the list of (request, key/value head, tile of 16 packed rows,
// kUnit keys); every block takes an equal, contiguous share of it, so a single
// long context keeps all SMs reading as well as many short ones do.  One warp
// copies K and V, page by page (TMA), as far ahead as there are stages, into
// the block's next tiles too; eight warps take an eighth of a unit's keys and keep a
// softmax state each.  The states are merged at the end of a tile, or of the
// block's part of it, and parts by paged_join_kernel.
//
// Bound by HBM: K and V are read once per 16 packed rows.  (mma.sync: 16 rows
// leave the tcgen05 tile of 128 empty, and the products are not the bound.)
// 64 ragged contexts up to 16K, 32 heads over 8, d 128: 335 to 345 us, 0.97 to 1.00
// of measured copy bandwidth; one context of 128K, 32 heads: 310 to 320 us, 1.00
// to 1.03; 128 contexts of 8K, 16 heads over 2, d 64: 91 us, 0.88.  A lone short
// context (777 keys) takes 12 us, launch included, a chain of latencies: lengths,
// page numbers, keys, merge.
template <int D, bool kHalf>
__global__ void __launch_bounds__(kThreads, 1)
paged_rows_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ RowsParams rp)
{
    using C = Cfg<D>;
    using Op = Operand<kHalf>;
    using Walk = rows::Walk<C::kUnit>;
    constexpr int kKeys = C::kKeys, kUnit = C::kUnit, kTiles8 = kKeys / 8, kSteps16 = kKeys / 16;
    extern __shared__ uint8_t smem_raw[];
    __shared__ long long s_scratch[kThreads / 32];
    __shared__ long long s_offset;
    __shared__ int s_req, s_abort;
    const AttnParams& p = rp.a;
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw_base);
    const uint32_t bar0 = base + C::kOffBar;
    auto bar_full = [&](int s) { return bar0 + 8u * s; };                          // copies -> products
    auto bar_empty = [&](int s) { return bar0 + 8u * (C::kStages + s); };          // products -> copies
    const uint32_t bar_given = bar0 + 8u * (2 * C::kStages);                       // every warp's state is written
    const uint32_t bar_taken = bar0 + 8u * (2 * C::kStages + 1);                   // and read
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    let_next_start();

    // ---- this block's share of the work
    const int per = (p.n + kThreads - 1) / kThreads;
    const int i0 = min(p.n, tid * per), i1 = min(p.n, i0 + per);
    long long mine = 0, total;
    for (int i = i0; i < i1; ++i) mine += Walk::cost(p, rp.range, i);
    const long long before = block_exclusive_sum(mine, s_scratch, &total);
    const int b = blockIdx.x;
    const Share share = share_of(total, gridDim.x, b);
    if (tid < 2) rp.ws.info[2 * b + tid].req = -1;
    if (share.count == 0) return;
    if (before <= share.start && share.start < before + mine) {
        long long x = share.start - before;
        int i = i0;
        for (long long c; x >= (c = Walk::cost(p, rp.range, i)); ++i) x -= c;
        s_req = i;
        s_offset = x;
    }
    if (tid == 0) {
        s_abort = 0;
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(bar_full(s), 1);
            mbar_init(bar_empty(s), kWarps);
        }
        mbar_init(bar_given, kWarps);
        mbar_init(bar_taken, kWarps);
        fence_mbar_init();
    }
    __syncthreads();
    Walk walk(p, rp.range, s_req, s_offset, share.count);
    if (walk.empty()) return;
    const WaitCtl wc{&s_abort, p.status, rp.wait_limit_ns};
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_inline(bar, parity & 1u, wc));
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if (warp > 0) return;
        // ------------------------------------------------------------ copies
        const int boxes = kUnit / rp.box_rows * C::kBoxes;      // at most 32: one for each lane
        const int box = lane / C::kBoxes, half = lane % C::kBoxes;
        const uint32_t box_dst = (uint32_t)(half * C::kBoxBytes + box * rp.box_rows * 128);
        if (lane == 0) {
            tma_prefetch_desc(&map_k);
            tma_prefetch_desc(&map_v);
        }
        bool ok = true;
        uint32_t n = 0;
        do {
            const int* table = p.table + (long long)walk.req * p.table_stride;
            const int keys = walk.keys(), kvh = walk.kvh(), u1 = walk.u1;
            auto page_at = [&](int u) {
                const int key = u * kUnit + box * rp.box_rows;
                return lane < boxes && u < u1 && key < keys ? table[page_index(key, p.page_size, p.page_shift)] : 0;
            };
            int page = page_at(walk.u0), then = page_at(walk.u0 + 1);
            for (int u = walk.u0; u < u1; ++u, ++n) {
                const int s = n % C::kStages;
                const int key = u * kUnit + box * rp.box_rows;
                const bool load = lane < boxes && key < keys;
                // a page outside the pool: a coordinate outside the map, which reads as zeros
                int coord = page;
                if (load && !page_ok(page, p.num_pages)) {
                    coord = p.num_pages;
                    atomicOr(p.status, kStatusBadPage);
                }
                const int off = key - page_index(key, p.page_size, p.page_shift) * p.page_size;
                page = then;
                then = page_at(u + 2);
                const uint32_t bytes = 2u * (uint32_t)__popc(__ballot_sync(0xffffffffu, load)) * rp.box_rows * 128u;
                if (!(ok = wait_all(bar_empty(s), (n / C::kStages) + 1u))) break;
                if (lane == 0) mbar_arrive_expect_tx(bar_full(s), bytes);
                __syncwarp();
                if (load) {
                    const uint32_t dst = base + 2 * s * C::kTileBytes + box_dst;
                    tma_load_4d(dst, &map_k, bar_full(s), 64 * half, off, kvh, coord);
                    tma_load_4d(dst + C::kTileBytes, &map_v, bar_full(s), 64 * half, off, kvh, coord);
                }
            }
        } while (ok && walk.next());
        // Every copy lands before the block's shared memory goes.
        volatile int dummy = 0;
        const WaitCtl drain{&dummy, p.status, 200000000ull};
        for (uint32_t x = n > C::kStages ? n - C::kStages : 0; x < n; ++x)
            mbar_wait_inline(bar_full(x % C::kStages), (x / C::kStages) & 1u, drain);
        return;
    }

    // -------------------------------------------------------------- products
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
    const int w = warp - 4, g = lane >> 2, t4 = lane & 3;
    // the warp's rows of a stage, kKeys w and on; 16-byte pieces swizzled by row
    const int k_row = (lane & 7) + ((lane >> 4) << 3), v_row = lane & 15;
    const uint32_t k_base = base + (uint32_t)(kKeys * w + k_row) * 128u;
    const uint32_t v_base = base + C::kTileBytes + (uint32_t)(kKeys * w + v_row) * 128u;
    auto load_q = [&](uint32_t (&qa)[D / 16][4]) {
        const int row0 = walk.row0(), rows = walk.rows(), kvh = walk.kvh();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = row0 + min(g + 8 * e, rows - 1);
            const int tok = row / p.group, head = kvh * p.group + (row - tok * p.group);
            const uint16_t* q = p.q + (long long)(walk.r.first + tok) * p.q_tok + (long long)head * p.q_head + t4 * 2;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qa[k][e] = *reinterpret_cast<const uint32_t*>(q + k * 16);
                qa[k][2 + e] = *reinterpret_cast<const uint32_t*>(q + k * 16 + 8);
            }
        }
    };
    uint32_t qa[D / 16][4];
    load_q(qa);
    uint32_t n = 0, merges = 0;
    bool ok = true, more = true;
    while (ok && more) {
        const int row0 = walk.row0(), rows = walk.rows(), kvh = walk.kvh(), keys = walk.keys();
        const Request r = walk.r;
        // the two rows of this thread: last key each attends to
        int lim[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int tok = (row0 + min(g + 8 * e, rows - 1)) / p.group;
            lim[e] = p.causal ? min(r.len, r.len - r.q + tok + 1) - 1 : r.len - 1;
        }
        // smallest limit of the tile
        const int lim_first = p.causal ? r.len - r.q + row0 / p.group : r.len - 1;

        struct {
            float m[2], l[2], acc[D / 8][4];     // 16 rows, of which a thread holds two
        } st;
        st.m[0] = st.m[1] = -INFINITY;
        st.l[0] = st.l[1] = 0.f;
#pragma unroll
        for (int x = 0; x < D / 8; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) st.acc[x][y] = 0.f;

        for (int u = walk.u0; u < walk.u1; ++u, ++n) {
            const int stage = n % C::kStages, key0 = u * kUnit + w * kKeys;
            if (!(ok = wait_all(bar_full(stage), n / C::kStages))) break;
            if (key0 >= keys) {
                if (lane == 0) mbar_arrive(bar_empty(stage));
                continue;
            }
            const uint32_t sK = k_base + 2 * stage * C::kTileBytes, sV = v_base + 2 * stage * C::kTileBytes;

            // ---- S = Q K^T: 16 rows x kKeys keys, even and odd k-steps apart
            float s[kTiles8][4], s2[kTiles8][4];
#pragma unroll
            for (int x = 0; x < kTiles8; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) s[x][y] = s2[x][y] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
#pragma unroll
                for (int z = 0; z < kSteps16; ++z) {
                    // matrices: keys 0-7 | 8-15, columns 16k..16k+7 | 16k+8..
                    uint32_t kb[4];
                    ldmatrix4(kb, sK + z * 2048 + (k >> 2) * C::kBoxBytes +
                                      (((2 * (k & 3) + ((lane >> 3) & 1)) ^ (k_row & 7)) << 4));
                    Op::mma(k & 1 ? s2[2 * z] : s[2 * z], qa[k], kb[0], kb[1]);
                    Op::mma(k & 1 ? s2[2 * z + 1] : s[2 * z + 1], qa[k], kb[2], kb[3]);
                }
            }
#pragma unroll
            for (int x = 0; x < kTiles8; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) s[x][y] += s2[x][y];

            // ---- softmax
            const bool masked = key0 + kKeys - 1 > lim_first;
#pragma unroll
            for (int x = 0; x < kTiles8; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    s[x][y] *= p.scale_log2;
                    if (masked && key0 + 8 * x + 2 * t4 + (y & 1) > lim[y >> 1]) s[x][y] = -INFINITY;
                }
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = max_nan(s[0][2 * e], s[0][2 * e + 1]);
#pragma unroll
                for (int x = 1; x < kTiles8; ++x) mx = max_nan(mx, max_nan(s[x][2 * e], s[x][2 * e + 1]));
                mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float m = max_nan(st.m[e], mx);
                alpha[e] = m == -INFINITY ? 1.f : ex2_approx(st.m[e] - m);
                st.m[e] = m;
                const float ref = m == -INFINITY ? 0.f : m - Op::kShift;
                float sum = 0.f;
#pragma unroll
                for (int x = 0; x < kTiles8; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float w = ex2_approx(s[x][2 * e + y] - ref);
                        s[x][2 * e + y] = w;
                        sum += w;
                    }
                st.l[e] = st.l[e] * alpha[e] + sum;
            }
            if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
                for (int x = 0; x < D / 8; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) st.acc[x][y] *= alpha[y >> 1];
            }
            // Weights in the operand type.  fp16's half step of 2^-11 stays.  bf16's
            // would show in O, so a weight is cut to its upper half and what that
            // leaves is rounded and multiplied too, for 1 % of a long decode's time:
            // 2^-16 of the weight is lost.  Cut, not rounded, and with the smallest
            // bf16 in place of a rest of 0, both parts have the weight's sign: an
            // infinity in V gives no NaN by the rest's 0 or -infinity.  (Against a
            // rounded upper half: long decodes the same, 64 contexts of up to 1153
            // keys, d 64, 77.7 -> 79.2 us.)  l sums the weights as they are.
            uint32_t pa[kSteps16][4], pr[kSteps16][4];
#pragma unroll
            for (int z = 0; z < kSteps16; ++z)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float w0 = s[2 * z + (i >> 1)][2 * (i & 1)], w1 = s[2 * z + (i >> 1)][2 * (i & 1) + 1];
                    if constexpr (kHalf) {
                        pa[z][i] = Op::pack(w0, w1);
                    } else {
                        const uint32_t b0 = __float_as_uint(w0), b1 = __float_as_uint(w1);
                        const float h0 = __uint_as_float(b0 & 0xffff0000u), h1 = __uint_as_float(b1 & 0xffff0000u);
                        pa[z][i] = __byte_perm(b0, b1, 0x7632);
                        pr[z][i] = Op::pack(fmaxf(w0 - h0, fminf(h0, kLeastBf16)), fmaxf(w1 - h1, fminf(h1, kLeastBf16)));
                    }
                }

            // ---- O += P V
            auto load_v = [&](uint32_t (&vb)[4], int z, int x) {
                // matrices: keys 0-7 | 8-15 of columns 16x.., then of 16x + 8..
                ldmatrix4_trans(vb, sV + z * 2048 + (x >> 2) * C::kBoxBytes +
                                        (((2 * (x & 3) + (lane >> 4)) ^ (v_row & 7)) << 4));
            };
            if (!masked) {
#pragma unroll
                for (int z = 0; z < kSteps16; ++z)
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        uint32_t vb[4];
                        load_v(vb, z, x);
                        Op::mma(st.acc[2 * x], pa[z], vb[0], vb[1]);
                        Op::mma(st.acc[2 * x + 1], pa[z], vb[2], vb[3]);
                        if constexpr (!kHalf) {
                            Op::mma(st.acc[2 * x], pr[z], vb[0], vb[1]);
                            Op::mma(st.acc[2 * x + 1], pr[z], vb[2], vb[3]);
                        }
                    }
            } else {
                // Rows of V behind the last key in use hold anything: cleared.
                // A weight of 0 does not hide an infinity or a NaN either, so
                // where rows see different keys and V holds one, the keys are
                // added one by one to the rows that see them.
#pragma unroll
                for (int z = 0; z < kSteps16; ++z) {
                    const int key16 = key0 + 16 * z;
                    const int valid = keys - key16 - 2 * t4;     // of this thread's keys 2 t4 + {0, 1, 8, 9}
                    const uint32_t lo = (valid > 0 ? 0xffffu : 0u) | (valid > 1 ? 0xffff0000u : 0u);
                    const uint32_t hi = (valid > 8 ? 0xffffu : 0u) | (valid > 9 ? 0xffff0000u : 0u);
                    bool odd = false;
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        uint32_t vb[4];
                        load_v(vb, z, x);
                        odd |= Op::nonfinite(vb[0] & lo) || Op::nonfinite(vb[1] & hi) || Op::nonfinite(vb[2] & lo) ||
                               Op::nonfinite(vb[3] & hi);
                    }
                    odd = __any_sync(0xffffffffu, odd);
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        uint32_t vb[4];
                        load_v(vb, z, x);
                        vb[0] &= lo;
                        vb[1] &= hi;
                        vb[2] &= lo;
                        vb[3] &= hi;
                        if (!odd) {
                            Op::mma(st.acc[2 * x], pa[z], vb[0], vb[1]);
                            Op::mma(st.acc[2 * x + 1], pa[z], vb[2], vb[3]);
                            if constexpr (!kHalf) {
                                Op::mma(st.acc[2 * x], pr[z], vb[0], vb[1]);
                                Op::mma(st.acc[2 * x + 1], pr[z], vb[2], vb[3]);
                            }
                            continue;
                        }
#pragma unroll 1
                        for (int key = 0; key < 16; ++key) {
                            const uint32_t sel = ((key & 7) >> 1) == t4 ? (key & 1 ? 0xffff0000u : 0x0000ffffu) : 0u;
                            const uint32_t lower = key < 8 ? sel : 0u, upper = key < 8 ? 0u : sel;
                            const uint32_t one[4] = {pa[z][0] & lower, pa[z][1] & lower, pa[z][2] & upper,
                                                     pa[z][3] & upper};
                            uint32_t rest[4] = {};
                            if constexpr (!kHalf) {
                                rest[0] = pr[z][0] & lower;
                                rest[1] = pr[z][1] & lower;
                                rest[2] = pr[z][2] & upper;
                                rest[3] = pr[z][3] & upper;
                            }
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                float d[4] = {0.f, 0.f, 0.f, 0.f};
                                Op::mma(d, one, vb[2 * y] & lower, vb[2 * y + 1] & upper);
                                if constexpr (!kHalf) Op::mma(d, rest, vb[2 * y] & lower, vb[2 * y + 1] & upper);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (key16 + key <= lim[e >> 1]) st.acc[2 * x + y][e] += d[e];
                            }
                        }
                    }
                }
            }
            __syncwarp();     // the stage may be written again
            if (lane == 0) mbar_arrive(bar_empty(stage));
        }
        if (!ok) break;

        // the next piece's queries are on their way while this one is merged
        const bool whole = walk.u0 == 0 && walk.u1 == walk.units;
        const int slot = 2 * b + (walk.u0 == 0);
        const PartInfo info{walk.req, kvh, row0, walk.u1 == walk.units};
        more = walk.next();
        if (more) load_q(qa);

        // ---- merge the eight warps, eight rows at a time: every warp writes
        // the rows in use of its state, then warp w sums row w over all of them.
        // Columns are swizzled by row, against bank conflicts.
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            st.l[e] += __shfl_xor_sync(0xffffffffu, st.l[e], 1);
            st.l[e] += __shfl_xor_sync(0xffffffffu, st.l[e], 2);
        }
        float* sums = reinterpret_cast<float*>(gbase + C::kOffSums);
        float* stat = reinterpret_cast<float*>(gbase + C::kOffStat);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (8 * e >= rows) break;
            if (!(ok = wait_all(bar_taken, merges + 1u))) break;
            if (8 * e + g < rows) {
                float* to = sums + (w * 8 + g) * D;
#pragma unroll
                for (int x = 0; x < D / 8; ++x)
                    *reinterpret_cast<float2*>(to + ((8 * x + 2 * t4) ^ (g << 3))) =
                        make_float2(st.acc[x][2 * e], st.acc[x][2 * e + 1]);
                if (t4 == 0) {
                    stat[w * 8 + g] = st.m[e];
                    stat[kWarps * 8 + w * 8 + g] = st.l[e];
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_given);
            if (!(ok = wait_all(bar_given, merges))) break;
            const int row = 8 * e + w;
            if (row < rows) {
                constexpr int kPer = D / 32;          // columns of a lane
                float m = -INFINITY, l = 0.f, out[kPer];
#pragma unroll
                for (int x = 0; x < kWarps; ++x) m = max_nan(m, stat[x * 8 + w]);
#pragma unroll
                for (int c = 0; c < kPer; ++c) out[c] = 0.f;
#pragma unroll
                for (int x = 0; x < kWarps; ++x) {
                    const float mx = stat[x * 8 + w];
                    // a state without keys is all 0 and adds nothing
                    const float f = mx == -INFINITY ? 0.f : ex2_approx(mx - m);
                    l += f * stat[kWarps * 8 + x * 8 + w];
                    const float* from = sums + (x * 8 + w) * D + ((kPer * lane) ^ (w << 3));
                    float v[kPer];
                    if constexpr (kPer == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(from);
                    else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(from);
#pragma unroll
                    for (int c = 0; c < kPer; ++c) out[c] += f * v[c];
                }
                const int col = kPer * lane;
                if (whole) {
                    store_row<kPer, kHalf>(p, r, kvh, row0 + row, col, out, m, l, Op::kShift);
                } else {
                    float* to = reinterpret_cast<float*>(part_columns<kRows>(rp.ws, slot, D, row, col)) + (col & 3);
                    if constexpr (kPer == 4) *reinterpret_cast<float4*>(to) = *reinterpret_cast<const float4*>(out);
                    else *reinterpret_cast<float2*>(to) = *reinterpret_cast<const float2*>(out);
                    if (lane == 0) {
                        rp.ws.ml[slot * 2 * kRows + row] = m;
                        rp.ws.ml[slot * 2 * kRows + kRows + row] = l;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_taken);
            ++merges;
        }
        if (!ok) break;
        if (!whole && w == 0 && lane == 0) rp.ws.info[slot] = info;
    }
}

}  // namespace rows
}  // namespace paged
}  // namespace ra
