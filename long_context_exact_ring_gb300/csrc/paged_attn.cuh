// paged_attn.cuh -- attention of new tokens over a paged key/value cache.
//
// Request i has len_i cached tokens, the last q_i of them new.  New token t
// sits at position len_i - q_i + t and attends to the keys c <= position
// (causal) or to all len_i keys:
//     s_c = scale <q, k_c>,  LSE = ln sum_c exp(s_c),  O = sum_c exp(s_c - LSE) v_c,
// and a row without keys gives O = 0, LSE = -inf.  Query head h reads
// key/value head h / group.  Key c lies in page block_table[i, c / page_size].
//
// The new tokens of a request that share a key/value head -- `group` query
// heads of each token -- are packed into rows r = token * group + head, so one
// pass over the keys serves all of them.
#pragma once

#include <cuda_fp16.h>

#include "paged_cache.cuh"

namespace ra {
namespace paged {

struct AttnParams {
    const uint16_t* q;
    long long q_tok, q_head;
    const uint16_t* kc;
    PoolLayout lk;
    const uint16_t* vc;
    PoolLayout lv;
    const int* table;
    long long table_stride;
    const int* seq_lens;
    const int* cu_q;
    uint16_t* o;
    long long o_tok, o_head;
    float* lse;              // [heads, tokens]
    int n, tokens, max_pages, num_pages, page_size, page_shift;   // page_shift < 0: not a power of two
    int kv_heads, group, causal;
    float scale_log2;
    uint32_t* status;
};

__device__ __forceinline__ Request load_request(const AttnParams& p, int i)
{
    return cut_request(p.cu_q[i], p.cu_q[i + 1], p.seq_lens[i], p.tokens, p.max_pages, p.page_size);
}

// The operand types: bf16 or fp16 products with fp32 accumulation.  kShift
// moves the reference of the exponentials: the weights 2^(x - m + kShift)
// are rounded to the operand type for the product with V, and fp16 would
// lose those below 2^-24; with the row maximum at 2^15 it keeps them down
// to 2^-39 of the largest.  bf16 has fp32's range and needs no shift.
template <bool kHalf> struct Operand;

template <> struct Operand<false> {
    static constexpr float kShift = 0.f;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
    static __device__ __forceinline__ bool nonfinite(uint32_t x)
    {
        return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
    }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

template <> struct Operand<true> {
    static constexpr float kShift = 15.f;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ bool nonfinite(uint32_t x)
    {
        return (x & 0x7c00u) == 0x7c00u || (x & 0x7c000000u) == 0x7c000000u;
    }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
    {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// max(a, b), NaN if either is: a NaN score has to reach its row's result.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take)
{
    const uint32_t bytes = take ? 16u : 0u;   // 0: the 16 bytes are filled with zeros, src is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// ---------------------------------------------------------------------------
// Parts.  A kernel cuts its list of (request, key/value head, tile of packed
// rows, keys) into equal, contiguous shares, one for each block.  A tile's
// keys are cut where one share ends and the next begins, so a block has at
// most two unfinished tiles: one that it takes over from the block before
// (part 0) and one that it leaves to the block behind (part 1).
// ---------------------------------------------------------------------------
constexpr int kMaxBlocks = 256;

struct PartInfo {
    int req;        // -1: no such part
    int kvh, row0;  // key/value head, first packed row
    int last;       // part 0 only: its tile ends in this block
};

struct Workspace {
    PartInfo* info;   // [blocks][2]
    float* ml;        // [blocks][2][2][tile rows] reference and sum of the exponentials
    float* acc;       // [blocks][2][D / 4][tile rows][4] sums, not normalized
};

// Workspace of a kernel with tiles of `rows` packed rows.
__host__ __device__ inline size_t workspace_bytes(int rows, int D)
{
    return (size_t)kMaxBlocks * 2 * (sizeof(PartInfo) + (2 * (size_t)rows + (size_t)rows * D) * 4);
}

__host__ __device__ inline Workspace workspace(void* base, int rows)
{
    Workspace w;
    w.info = static_cast<PartInfo*>(base);
    w.ml = reinterpret_cast<float*>(w.info + 2 * kMaxBlocks);
    w.acc = w.ml + (size_t)kMaxBlocks * 2 * 2 * rows;
    return w;
}

// Where four columns of a part's row lie: the rows of a tile are neighbours, so
// that lanes which hold a row each write whole lines.
__device__ __forceinline__ float4* part_columns(const Workspace& ws, int slot, int tile_rows, int D, int row, int col)
{
    return reinterpret_cast<float4*>(ws.acc) + ((size_t)slot * (D / 4) + col / 4) * tile_rows + row;
}

// Which requests a kernel serves: those with more than `above` and at most
// `upto` packed rows.
struct RowRange {
    int above, upto;
    __device__ __forceinline__ bool has(int rows) const { return rows > above && rows <= upto; }
};

// Writes kPer columns of a finished row.
template <int kPer, bool kHalf>
__device__ __forceinline__ void store_row(const AttnParams& p, const Request& r, int kvh, int packed, int col,
                                          const float (&out)[kPer], float m, float l, float shift)
{
    using Op = Operand<kHalf>;
    // no key, or none with a weight: O = 0, LSE = -inf
    const float inv = m == -INFINITY ? 0.f : 1.f / l;
    const int tok = packed / p.group, head = kvh * p.group + (packed - tok * p.group);
    uint16_t* dst = p.o + (long long)(r.first + tok) * p.o_tok + (long long)head * p.o_head + col;
    uint32_t pk[kPer / 2];
#pragma unroll
    for (int c = 0; c < kPer / 2; ++c) pk[c] = Op::pack(out[2 * c] * inv, out[2 * c + 1] * inv);
    if constexpr (kPer == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    else *reinterpret_cast<uint2*>(dst) = make_uint2(pk[0], pk[1]);
    if (col == 0)
        p.lse[(long long)head * p.tokens + r.first + tok] =
            m == -INFINITY ? -INFINITY : (m - shift + log2f(l)) * 0.69314718055994531f;
}

// Launches that follow one another without a gap: a kernel lets the next one
// start as soon as SMs are free, and the next one waits, where it needs the
// results, for the kernels before it to be over.  Every kernel waits at least
// at its end, so that the last one's end is the end of all.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Joins the parts of a tile that several blocks had a share of: the block
// that began it, then those behind it, in order -- the sum does not depend
// on which finished first.  A tile's rows come in halves of kHalfRows, of
// which the first `used` hold packed rows.  Joins rows 16 slice .. 16 slice +
// 15 of the tile that block b began and did not finish.
template <int D, bool kHalf, int kTileRows, int kHalfRows>
__device__ __forceinline__ void join_part(const AttnParams& p, const Workspace& ws, int blocks, int b, int slice,
                                          int used, float shift)
{
    const PartInfo info = ws.info[2 * b + 1];
    if (info.req < 0) return;
    constexpr int kPer = 16 * D / 256;
    const int row = slice * 16 + threadIdx.x % 16, col = threadIdx.x / 16 * kPer;
    const Request r = load_request(p, info.req);
    const int packed = info.row0 + row / kHalfRows * used + row % kHalfRows;
    if (row % kHalfRows >= used || packed >= r.q * p.group) return;
    float m = -INFINITY, l = 0.f, out[kPer];
#pragma unroll
    for (int c = 0; c < kPer; ++c) out[c] = 0.f;
    for (int x = b; x < blocks; ++x) {
        const int slot = x == b ? 2 * b + 1 : 2 * x;
        bool last = false;
        if (x != b) {
            const PartInfo next = ws.info[slot];
            if (next.req < 0) continue;      // a block without work
            last = next.last;
        }
        const float mx = ws.ml[(size_t)slot * 2 * kTileRows + row];
        const float lx = ws.ml[(size_t)slot * 2 * kTileRows + kTileRows + row];
        float v[kPer];
#pragma unroll
        for (int c = 0; c < kPer; c += 4)
            *reinterpret_cast<float4*>(v + c) = *part_columns(ws, slot, kTileRows, D, row, col + c);
        if (mx != -INFINITY) {
            const float to = max_nan(m, mx), fa = ex2_approx(m - to), fb = ex2_approx(mx - to);
            m = to;
            l = l * fa + lx * fb;
#pragma unroll
            for (int c = 0; c < kPer; ++c) out[c] = out[c] * fa + v[c] * fb;
        }
        if (last) break;
    }
    store_row<kPer, kHalf>(p, r, info.kvh, packed, col, out, m, l, shift);
}

// The two kernels' tiles (paged_rows_kernel's, paged_tiles_kernel's): rows of
// a tile, rows of its halves, shift of the reference.
constexpr int kRowsTile = 16, kBigTile = 256, kBigHalf = 128;
template <bool kHalf> constexpr float kBigShift = kHalf ? 7.f : 0.f;
constexpr int kBigSlices = kBigTile / 16;

// Slices 0 .. kBigSlices - 1 of the large tiles, then the small ones.
template <int D, bool kHalf>
__global__ void __launch_bounds__(256)
paged_join_kernel(const AttnParams p, const Workspace rows, const Workspace big, int blocks, int used, int first_slice)
{
    wait_for_previous();
    const int slice = blockIdx.y + first_slice;
    if (slice == kBigSlices)
        join_part<D, kHalf, kRowsTile, kRowsTile>(p, rows, blocks, blockIdx.x, 0, kRowsTile, Operand<kHalf>::kShift);
    else
        join_part<D, kHalf, kBigTile, kBigHalf>(p, big, blocks, blockIdx.x, slice, used, kBigShift<kHalf>);
}

namespace rows {

constexpr int kRows = kRowsTile;   // packed rows of a tile: one m16n8k16 operand
constexpr int kKeys = 16;        // keys of a warp's step
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = kKeys * kWarps;   // keys of a block's step, and of the smallest piece of work

template <int D>
struct Cfg {
    static constexpr int kChunkBytes = kKeys * D * 2;              // a warp's K (or V) of one step
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kWarpBytes = 2 * kChunkBytes * kStages;
    static constexpr int kSmemBytes = kWarps * kWarpBytes;
    static_assert(kWarpBytes >= kRows * D * 4 + 2 * kRows * 4, "a warp's state fits over its stages");
};

// One warp's running state of a tile: 16 rows, of which a thread holds two.
template <int D>
struct State {
    float m[2], l[2];
    float acc[D / 8][4];
};

// The work is the list of (request, key/value head, tile of 16 packed rows,
// 128 keys); every block takes an equal, contiguous share of it, so a single
// long context keeps all SMs reading as well as many short ones do.  Every
// warp streams its own 16 keys out of each 128 through its own ring of
// stages (asynchronous copies, no barrier between warps) and keeps its own
// softmax state; the states of the eight warps are merged at the end of a
// tile, or of the block's part of it, and parts by paged_join_kernel.
//
// Bound by HBM: K and V are read once per 16 packed rows.
template <int D, bool kHalf>
__global__ void __launch_bounds__(kThreads, 1) paged_rows_kernel(const AttnParams p, const Workspace ws, const RowRange range)
{
    using C = Cfg<D>;
    using Op = Operand<kHalf>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ long long s_scratch[kWarps + 1];
    __shared__ long long s_offset;
    __shared__ int s_req;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t4 = lane & 3;
    uint8_t* my = smem_raw + warp * C::kWarpBytes;
    const uint32_t s_my = smem_u32(my);
    let_next_start();

    // ---- this block's share of the work
    auto tiles_of = [&](const Request& r) { return (r.q * p.group + kRows - 1) / kRows; };
    auto units_of = [&](const Request& r) { return max(1, (r.len + kUnit - 1) / kUnit); };
    auto work_of = [&](int i) {
        const Request r = load_request(p, i);
        return range.has(r.q * p.group) ? (long long)tiles_of(r) * p.kv_heads * units_of(r) : 0ll;
    };
    const int per = (p.n + kThreads - 1) / kThreads;
    const int i0 = min(p.n, tid * per), i1 = min(p.n, i0 + per);
    long long mine = 0, total;
    for (int i = i0; i < i1; ++i) mine += work_of(i);
    const long long before = block_exclusive_sum(mine, s_scratch, &total);
    const int G = gridDim.x, b = blockIdx.x;
    const Share share = share_of(total, G, b);
    const long long start = share.start;
    long long left = share.count;
    if (tid < 2) ws.info[2 * b + tid].req = -1;
    if (left == 0) return;
    if (before <= start && start < before + mine) {
        long long x = start - before;
        int i = i0;
        for (long long c; x >= (c = work_of(i)); ++i) x -= c;
        s_req = i;
        s_offset = x;
    }
    __syncthreads();
    int req = s_req;
    long long offset = s_offset;                                     // units into the request

    while (true) {
        const Request r = load_request(p, req);
        const int tiles = tiles_of(r), units = units_of(r);
        const int item = (int)(offset / units);
        const int u0 = (int)(offset - (long long)item * units);
        const int u1 = (int)min((long long)units, u0 + left);
        const int kvh = item / tiles, row0 = (item - kvh * tiles) * kRows;
        const int rows = min(kRows, r.q * p.group - row0);
        const int* table = p.table + (long long)req * p.table_stride;

        // the two rows of this thread: last key each attends to
        int lim[2];
        long long q_off[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = row0 + min(g + 8 * e, rows - 1);
            const int tok = row / p.group, head = kvh * p.group + (row - tok * p.group);
            lim[e] = p.causal ? min(r.len, r.len - r.q + tok + 1) - 1 : r.len - 1;
            q_off[e] = (long long)(r.first + tok) * p.q_tok + (long long)head * p.q_head;
        }
        const int tok_first = row0 / p.group, tok_last = (row0 + rows - 1) / p.group;
        const int lim_first = p.causal ? r.len - r.q + tok_first : r.len - 1;   // smallest limit of the tile
        const int keys = min(u1 * kUnit, p.causal ? r.len - r.q + tok_last + 1 : r.len);

        // ---- copies: page sizes are multiples of 8, so 8 keys share a page;
        // the page numbers are fetched one step ahead of the copies
        constexpr int kPieces = D / 8;                   // 16-byte pieces of a row
        constexpr int kRowsPerOp = 32 / kPieces;
        auto fetch_pages = [&](int key0, int (&pg)[2]) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
                pg[hf] = key0 + 8 * hf < keys ? table[page_index(key0 + 8 * hf, p.page_size, p.page_shift)] : 0;
        };
        auto copy = [&](int key0, int stage, const int (&pg)[2]) {
            long long kb[2], vb[2];
            bool ok[2], bad = false;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int key = key0 + 8 * hf;
                ok[hf] = key < keys;
                if (!page_ok(pg[hf], p.num_pages)) {
                    ok[hf] = false;
                    bad = true;
                }
                const int off = key - page_index(key, p.page_size, p.page_shift) * p.page_size;
                kb[hf] = ok[hf] ? row_offset(p.lk, pg[hf], off, kvh) : 0;
                vb[hf] = ok[hf] ? row_offset(p.lv, pg[hf], off, kvh) : 0;
            }
            if (bad && lane == 0) atomicOr(p.status, kStatusBadPage);
            const uint32_t sK = s_my + stage * 2 * C::kChunkBytes, sV = sK + C::kChunkBytes;
#pragma unroll
            for (int x = 0; x < kKeys / kRowsPerOp; ++x) {
                const int row = x * kRowsPerOp + lane / kPieces, piece = lane % kPieces;
                const int hf = row >> 3, in = row & 7;
                const bool take = ok[hf] && key0 + row < r.len;
                const uint32_t dst = (uint32_t)(row * D * 2 + ((piece ^ in) << 4));
                cp_async16(sK + dst, p.kc + kb[hf] + (take ? in * p.lk.st : 0) + piece * 8, take);
                cp_async16(sV + dst, p.vc + vb[hf] + (take ? in * p.lv.st : 0) + piece * 8, take);
            }
        };
        const int first = u0 * kUnit + warp * kKeys;
        int pg[2];
        fetch_pages(first, pg);
#pragma unroll
        for (int x = 0; x < C::kStages - 1; ++x) {
            const int key0 = first + x * kUnit;
            if (key0 < keys) copy(key0, x, pg);
            cp_async_commit();
            fetch_pages(key0 + kUnit, pg);
        }

        uint32_t qa[D / 16][4];
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                qa[k][e] = *reinterpret_cast<const uint32_t*>(p.q + q_off[e] + k * 16 + t4 * 2);
                qa[k][2 + e] = *reinterpret_cast<const uint32_t*>(p.q + q_off[e] + k * 16 + 8 + t4 * 2);
            }
        }

        State<D> st;
        st.m[0] = st.m[1] = -INFINITY;
        st.l[0] = st.l[1] = 0.f;
#pragma unroll
        for (int x = 0; x < D / 8; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) st.acc[x][y] = 0.f;

        int stage = 0;
        for (int key0 = first; key0 < keys; key0 += kUnit) {
            {
                const int ahead = key0 + (C::kStages - 1) * kUnit;
                if (ahead < keys) copy(ahead, stage == 0 ? C::kStages - 1 : stage - 1, pg);
                cp_async_commit();
                fetch_pages(ahead + kUnit, pg);
            }
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

        // ---- merge the eight warps
        cp_async_wait<0>();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            st.l[e] += __shfl_xor_sync(0xffffffffu, st.l[e], 1);
            st.l[e] += __shfl_xor_sync(0xffffffffu, st.l[e], 2);
        }
        __syncwarp();
        float* mo = reinterpret_cast<float*>(my);
#pragma unroll
        for (int x = 0; x < D / 8; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float2*>(mo + (g + 8 * e) * D + 8 * x + 2 * t4) =
                    make_float2(st.acc[x][2 * e], st.acc[x][2 * e + 1]);
        if (t4 == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mo[kRows * D + g + 8 * e] = st.m[e];
                mo[kRows * D + kRows + g + 8 * e] = st.l[e];
            }
        }
        __syncthreads();
        constexpr int kPer = kRows * D / kThreads;       // columns of a thread
        const int row = tid / (D / kPer), col = tid % (D / kPer) * kPer;
        auto part = [&](int w) { return reinterpret_cast<const float*>(smem_raw + w * C::kWarpBytes); };
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = max_nan(m, part(w)[kRows * D + row]);
        float l = 0.f, out[kPer];
#pragma unroll
        for (int c = 0; c < kPer; ++c) out[c] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = part(w)[kRows * D + row];
            if (mw == -INFINITY) continue;           // no key of this row
            const float f = ex2_approx(mw - m);
            l += f * part(w)[kRows * D + kRows + row];
#pragma unroll
            for (int c = 0; c < kPer; ++c) out[c] += f * part(w)[row * D + col + c];
        }
        if (u0 == 0 && u1 == units) {
            if (row < rows) store_row<kPer, kHalf>(p, r, kvh, row0 + row, col, out, m, l, Op::kShift);
        } else {
            const int slot = 2 * b + (u0 == 0);
#pragma unroll
            for (int c = 0; c < kPer; c += 4)
                *part_columns(ws, slot, kRows, D, row, col + c) = make_float4(out[c], out[c + 1], out[c + 2], out[c + 3]);
            if (col == 0) {
                ws.ml[slot * 2 * kRows + row] = m;
                ws.ml[slot * 2 * kRows + kRows + row] = l;
            }
            if (tid == 0) ws.info[slot] = PartInfo{req, kvh, row0, u1 == units};
        }
        left -= u1 - u0;
        if (left == 0) break;
        offset += u1 - u0;
        if (offset == (long long)tiles * p.kv_heads * units) {
            offset = 0;
            do ++req;
            while (work_of(req) == 0);       // some later request has the work that is left
        }
        __syncthreads();                     // the states are read before the stages are filled again
    }
}

}  // namespace rows
}  // namespace paged
}  // namespace ra
