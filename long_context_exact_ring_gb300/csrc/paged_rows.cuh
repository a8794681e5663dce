// paged_rows.cuh -- attention of few new tokens over a paged cache: the form
// of paged_attn_fwd for decode steps.
#pragma once

#include "paged_attn.cuh"

namespace ra {
namespace paged {
namespace rows {

constexpr int kRows = kRowsTile;        // packed rows of a tile: one m16n8k16 operand
constexpr int kKeys = 16;               // keys of a warp's step
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = kKeys * kWarps;   // keys of a block's step, and of the smallest piece of work

template <int D>
struct Cfg {
    static constexpr int kChunkBytes = kKeys * D * 2;              // a warp's K (or V) of one step
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kWarpBytes = 2 * kChunkBytes * kStages;
    static constexpr int kStateBytes = kRows * D * 4 + 2 * kRows * 4;
    static constexpr int kOffMerge = kWarps * kWarpBytes;
    static constexpr int kSmemBytes = kOffMerge + kWarps / 2 * kStateBytes;
};

// What a tile costs beside its keys, in units: the states of eight warps are
// merged and the results written, about 3 us against 1.5 us for a unit.  64
// ragged contexts up to 16K: 365 us without it, 355 with 1, 340 with 2, 343 with 3.
constexpr int kExtra = 2;

// A block's place in its share: units [u0, u1) of 128 keys of a tile.
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

// The work is the list of (request, key/value head, tile of 16 packed rows,
// 128 keys); every block takes an equal, contiguous share of it, so a single
// long context keeps all SMs reading as well as many short ones do.  Every
// warp streams its own 16 keys out of each 128 through its own ring of
// stages (asynchronous copies, no barrier between warps) and keeps its own
// softmax state; the states of the eight warps are merged in pairs at the end
// of a tile, or of the block's part of it, and parts by paged_join_kernel.  A
// warp's copies run ahead of its products into the block's next tile, so the
// SM goes on reading while states are merged and results are written.
//
// Bound by HBM: K and V are read once per 16 packed rows.
template <int D, bool kHalf>
__global__ void __launch_bounds__(kThreads, 1) paged_rows_kernel(const AttnParams p, const Workspace ws, const RowRange range)
{
    using C = Cfg<D>;
    using Op = Operand<kHalf>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ long long s_scratch[kWarps];
    __shared__ long long s_offset;
    __shared__ int s_req;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const uint32_t s_my = smem_u32(smem_raw) + warp * C::kWarpBytes;
    let_next_start();

    // ---- this block's share of the work
    const int per = (p.n + kThreads - 1) / kThreads;
    const int i0 = min(p.n, tid * per), i1 = min(p.n, i0 + per);
    long long mine = 0, total;
    for (int i = i0; i < i1; ++i) mine += Walk::cost(p, range, i);
    const long long before = block_exclusive_sum(mine, s_scratch, &total);
    const int b = blockIdx.x;
    const Share share = share_of(total, gridDim.x, b);
    if (tid < 2) ws.info[2 * b + tid].req = -1;
    if (share.count == 0) return;
    if (before <= share.start && share.start < before + mine) {
        long long x = share.start - before;
        int i = i0;
        for (long long c; x >= (c = Walk::cost(p, range, i)); ++i) x -= c;
        s_req = i;
        s_offset = x;
    }
    __syncthreads();
    Walk walk(p, range, s_req, s_offset, share.count);
    if (walk.empty()) return;

    // ---- copies, ahead of the products.  Page sizes are multiples of 8, so 8
    // keys share a page.  A lane holds the page of one half of one of 16 steps,
    // and another for the 16 behind those, so no copy waits for its page.
    constexpr int kPieces = D / 8;                   // 16-byte pieces of a row
    constexpr int kRowsPerOp = 32 / kPieces;
    Walk ahead = walk;
    int a_key, a_keys, a_kvh, a_step, a_stage = 0, page_now, page_then;
    bool a_more = true;
    const int* a_table;
    auto fetch_page = [&](int key) {
        key += (lane >> 1) * kUnit + (lane & 1) * 8;
        return key < a_keys ? __ldg(a_table + page_index(key, p.page_size, p.page_shift)) : 0;
    };
    auto enter = [&]() {
        a_key = ahead.u0 * kUnit + warp * kKeys;
        a_keys = ahead.keys();
        a_kvh = ahead.kvh();
        a_table = p.table + (long long)ahead.req * p.table_stride;
        a_step = 0;
        page_now = fetch_page(a_key);
        page_then = fetch_page(a_key + 16 * kUnit);
    };
    auto copy_next = [&]() {
        while (a_more && a_key >= a_keys) {
            a_more = ahead.next();
            if (a_more) enter();
        }
        if (a_more) {
            long long kb[2], vb[2];
            bool ok[2], bad = false;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int key = a_key + 8 * hf, page = __shfl_sync(0xffffffffu, page_now, 2 * a_step + hf);
                ok[hf] = key < a_keys;
                if (!page_ok(page, p.num_pages)) {
                    ok[hf] = false;
                    bad = true;
                }
                const int off = key - page_index(key, p.page_size, p.page_shift) * p.page_size;
                kb[hf] = ok[hf] ? row_offset(p.lk, page, off, a_kvh) : 0;
                vb[hf] = ok[hf] ? row_offset(p.lv, page, off, a_kvh) : 0;
            }
            if (bad && lane == 0) atomicOr(p.status, kStatusBadPage);
            const uint32_t sK = s_my + a_stage * 2 * C::kChunkBytes, sV = sK + C::kChunkBytes;
#pragma unroll
            for (int x = 0; x < kKeys / kRowsPerOp; ++x) {
                const int row = x * kRowsPerOp + lane / kPieces, piece = lane % kPieces;
                const int hf = row >> 3, in = row & 7;
                const bool take = ok[hf] && a_key + row < ahead.r.len;
                const uint32_t dst = (uint32_t)(row * D * 2 + ((piece ^ in) << 4));
                cp_async16(sK + dst, p.kc + kb[hf] + (take ? in * p.lk.st : 0) + piece * 8, take);
                cp_async16(sV + dst, p.vc + vb[hf] + (take ? in * p.lv.st : 0) + piece * 8, take);
            }
            a_stage = a_stage + 1 == C::kStages ? 0 : a_stage + 1;
            a_key += kUnit;
            if (++a_step == 16) {
                a_step = 0;
                page_now = page_then;
                page_then = fetch_page(a_key + 16 * kUnit);
            }
        }
        cp_async_commit();
    };
    enter();
#pragma unroll 1
    for (int x = 0; x < C::kStages - 1; ++x) copy_next();

    int stage = 0;
    do {
        const int row0 = walk.row0(), rows = walk.rows(), kvh = walk.kvh();
        const Request r = walk.r;
        const int keys = walk.keys();
        // the two rows of this thread: last key each attends to
        int lim[2];
        uint32_t qa[D / 16][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = row0 + min(g + 8 * e, rows - 1);
            const int tok = row / p.group, head = kvh * p.group + (row - tok * p.group);
            lim[e] = p.causal ? min(r.len, r.len - r.q + tok + 1) - 1 : r.len - 1;
            const uint16_t* q = p.q + (long long)(r.first + tok) * p.q_tok + (long long)head * p.q_head + t4 * 2;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qa[k][e] = *reinterpret_cast<const uint32_t*>(q + k * 16);
                qa[k][2 + e] = *reinterpret_cast<const uint32_t*>(q + k * 16 + 8);
            }
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

        for (int key0 = walk.u0 * kUnit + warp * kKeys; key0 < keys; key0 += kUnit) {
            copy_next();
            cp_async_wait<C::kStages - 1>();
            __syncwarp();
            const uint32_t sK = s_my + stage * 2 * C::kChunkBytes, sV = sK + C::kChunkBytes;
            stage = stage + 1 == C::kStages ? 0 : stage + 1;

            // ---- S = Q K^T: 16 rows x 16 keys
            float s[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) s[x][y] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                // matrices: keys 0-7 | 8-15, columns 16k..16k+7 | 16k+8..
                const int row = (lane & 7) + ((lane >> 4) << 3), piece = 2 * k + ((lane >> 3) & 1);
                uint32_t b[4];
                ldmatrix4(b, sK + row * D * 2 + ((piece ^ (row & 7)) << 4));
                Op::mma(s[0], qa[k], b[0], b[1]);
                Op::mma(s[1], qa[k], b[2], b[3]);
            }

            // ---- softmax
            const bool masked = key0 + kKeys - 1 > lim_first;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    s[x][y] *= p.scale_log2;
                    if (masked && key0 + 8 * x + 2 * t4 + (y & 1) > lim[y >> 1]) s[x][y] = -INFINITY;
                }
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = max_nan(max_nan(s[0][2 * e], s[0][2 * e + 1]), max_nan(s[1][2 * e], s[1][2 * e + 1]));
                mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float m = max_nan(st.m[e], mx);
                alpha[e] = m == -INFINITY ? 1.f : ex2_approx(st.m[e] - m);
                st.m[e] = m;
                const float ref = m == -INFINITY ? 0.f : m - Op::kShift;
                float sum = 0.f;
#pragma unroll
                for (int x = 0; x < 2; ++x)
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
            // Weights rounded to the operand type (half a step of 2^-9 or
            // 2^-12 each); l sums them unrounded.
            uint32_t pa[4];
            pa[0] = Op::pack(s[0][0], s[0][1]);
            pa[1] = Op::pack(s[0][2], s[0][3]);
            pa[2] = Op::pack(s[1][0], s[1][1]);
            pa[3] = Op::pack(s[1][2], s[1][3]);

            // ---- O += P V
            bool odd = false;
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
                // matrices: keys 0-7 | 8-15 of columns 16x.., then of 16x + 8..
                const int row = lane & 15, piece = 2 * x + (lane >> 4);
                uint32_t b[4];
                ldmatrix4_trans(b, sV + row * D * 2 + ((piece ^ (row & 7)) << 4));
                if (!masked) {
                    Op::mma(st.acc[2 * x], pa, b[0], b[1]);
                    Op::mma(st.acc[2 * x + 1], pa, b[2], b[3]);
                } else {
                    odd |= Op::nonfinite(b[0]) || Op::nonfinite(b[1]) || Op::nonfinite(b[2]) || Op::nonfinite(b[3]);
                }
            }
            if (masked) {
                // A weight of 0 does not hide an infinity or a NaN in V, so
                // where rows see different keys and V holds one, the keys are
                // added one by one to the rows that see them.
                if (!__any_sync(0xffffffffu, odd)) {
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const int row = lane & 15, piece = 2 * x + (lane >> 4);
                        uint32_t b[4];
                        ldmatrix4_trans(b, sV + row * D * 2 + ((piece ^ (row & 7)) << 4));
                        Op::mma(st.acc[2 * x], pa, b[0], b[1]);
                        Op::mma(st.acc[2 * x + 1], pa, b[2], b[3]);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const int row = lane & 15, piece = 2 * x + (lane >> 4);
                        uint32_t b[4];
                        ldmatrix4_trans(b, sV + row * D * 2 + ((piece ^ (row & 7)) << 4));
#pragma unroll 1
                        for (int key = 0; key < kKeys; ++key) {
                            const uint32_t sel = ((key & 7) >> 1) == t4 ? (key & 1 ? 0xffff0000u : 0x0000ffffu) : 0u;
                            const uint32_t lo = key < 8 ? sel : 0u, hi = key < 8 ? 0u : sel;
                            const uint32_t a[4] = {pa[0] & lo, pa[1] & lo, pa[2] & hi, pa[3] & hi};
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                float d[4] = {0.f, 0.f, 0.f, 0.f};
                                Op::mma(d, a, b[2 * y] & lo, b[2 * y + 1] & hi);
#pragma unroll
                                for (int z = 0; z < 4; ++z)
                                    if (key0 + key <= lim[z >> 1]) st.acc[2 * x + y][z] += d[z];
                            }
                        }
                    }
                }
            }
            __syncwarp();     // the stage may be written again
        }

        // ---- merge the eight warps: 4-7 into 0-3, 2-3 into 0-1, 1 into 0
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            st.l[e] += __shfl_xor_sync(0xffffffffu, st.l[e], 1);
            st.l[e] += __shfl_xor_sync(0xffffffffu, st.l[e], 2);
        }
#pragma unroll 1
        for (int half = kWarps / 2; half > 0; half >>= 1) {
            float* state = reinterpret_cast<float*>(smem_raw + C::kOffMerge + (warp & (half - 1)) * C::kStateBytes);
            float4* acc = reinterpret_cast<float4*>(state) + lane;
            float* ml = state + kRows * D;
            __syncthreads();          // the states are read
            if (warp >= half && warp < 2 * half) {
#pragma unroll
                for (int x = 0; x < D / 8; ++x)
                    acc[32 * x] = make_float4(st.acc[x][0], st.acc[x][1], st.acc[x][2], st.acc[x][3]);
                if (t4 == 0) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        ml[g + 8 * e] = st.m[e];
                        ml[kRows + g + 8 * e] = st.l[e];
                    }
                }
            }
            __syncthreads();
            if (warp < half) {
                float mine[2], other[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mo = ml[g + 8 * e];
                    const float m = max_nan(st.m[e], mo);
                    // a state without keys is all 0 and adds nothing
                    mine[e] = st.m[e] == -INFINITY ? 0.f : ex2_approx(st.m[e] - m);
                    other[e] = mo == -INFINITY ? 0.f : ex2_approx(mo - m);
                    st.m[e] = m;
                    st.l[e] = st.l[e] * mine[e] + ml[kRows + g + 8 * e] * other[e];
                }
#pragma unroll
                for (int x = 0; x < D / 8; ++x) {
                    const float4 v = acc[32 * x];
                    st.acc[x][0] = st.acc[x][0] * mine[0] + v.x * other[0];
                    st.acc[x][1] = st.acc[x][1] * mine[0] + v.y * other[0];
                    st.acc[x][2] = st.acc[x][2] * mine[1] + v.z * other[1];
                    st.acc[x][3] = st.acc[x][3] * mine[1] + v.w * other[1];
                }
            }
        }
        if (warp == 0) {
            const bool whole = walk.u0 == 0 && walk.u1 == walk.units;
            const int slot = 2 * b + (walk.u0 == 0);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = g + 8 * e;
                if (whole) {
                    if (row >= rows) continue;
                    // no key, or none with a weight: O = 0, LSE = -inf
                    const float inv = st.m[e] == -INFINITY ? 0.f : 1.f / st.l[e];
                    const int tok = (row0 + row) / p.group, head = kvh * p.group + (row0 + row - tok * p.group);
                    uint16_t* dst = p.o + (long long)(r.first + tok) * p.o_tok + (long long)head * p.o_head + 2 * t4;
#pragma unroll
                    for (int x = 0; x < D / 8; ++x)
                        *reinterpret_cast<uint32_t*>(dst + 8 * x) =
                            Op::pack(st.acc[x][2 * e] * inv, st.acc[x][2 * e + 1] * inv);
                    if (t4 == 0)
                        p.lse[(long long)head * p.tokens + r.first + tok] =
                            st.m[e] == -INFINITY ? -INFINITY
                                                 : (st.m[e] - Op::kShift + log2f(st.l[e])) * 0.69314718055994531f;
                } else {
#pragma unroll
                    for (int x = 0; x < D / 8; ++x)
                        reinterpret_cast<float2*>(part_columns(ws, slot, kRows, D, row, 8 * x + 2 * t4))[t4 & 1] =
                            make_float2(st.acc[x][2 * e], st.acc[x][2 * e + 1]);
                    if (t4 == 0) {
                        ws.ml[slot * 2 * kRows + row] = st.m[e];
                        ws.ml[slot * 2 * kRows + kRows + row] = st.l[e];
                    }
                }
            }
            if (!whole && lane == 0) ws.info[slot] = PartInfo{walk.req, kvh, row0, walk.u1 == walk.units};
        }
    } while (walk.next());
}

}  // namespace rows
}  // namespace paged
}  // namespace ra
