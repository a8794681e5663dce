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
constexpr int kMaxBlocks = 160;    // one to an SM: 152
constexpr int kJoinThreads = 256;
static_assert(kMaxBlocks <= kJoinThreads, "a thread of the join to each block");

struct PartInfo {
    int req;        // -1: no such part
    int kvh, row0;  // key/value head, first packed row
    int last;       // part 0 only: its tile ends in this block
};

struct Workspace {
    PartInfo* info;   // [blocks][2]
    float* ml;        // [blocks][2][2][tile rows] reference and sum of the exponentials
    float* acc;       // [blocks][2][tile rows x D] sums, not normalized (part_columns)
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

// Where four columns of a part's row lie.  In a large tile the rows are
// neighbours, as a lane that writes holds a row; in a small one the columns, as
// a warp holds a row: either way a warp writes whole lines.
template <int kTileRows>
__device__ __forceinline__ float4* part_columns(const Workspace& ws, int slot, int D, int row, int col)
{
    float4* part = reinterpret_cast<float4*>(ws.acc) + (size_t)slot * kTileRows * (D / 4);
    return part + (kTileRows == 16 ? row * (D / 4) + col / 4 : col / 4 * kTileRows + row);
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
    else if constexpr (kPer == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(pk[0], pk[1]);
    else *reinterpret_cast<uint32_t*>(dst) = pk[0];
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

// The two kernels' tiles (paged_rows_kernel's, paged_tiles_kernel's): rows of
// a tile, rows of its halves, shift of the reference; slices of a tile that
// are joined by a block each.
constexpr int kRowsTile = 16, kBigTile = 256, kBigHalf = 128;
template <bool kHalf> constexpr float kBigShift = kHalf ? 7.f : 0.f;
constexpr int kRowsSlices = 4, kBigSlices = 16;

struct JoinShared {
    int slot[kMaxBlocks], base[kJoinThreads / 32], end;
    alignas(16) float m[kMaxBlocks][16];
    float l[kMaxBlocks][16];
};

// The parts of the tile that block b began and did not finish: this block's,
// then those of the blocks behind it up to the one that ends the tile (a block
// without work has none), with the references and sums of kRows of its rows.
// Returns their number.
template <int kTileRows, int kRows>
__device__ __forceinline__ int list_parts(const Workspace& ws, int blocks, int b, int row0, JoinShared& s)
{
    const int tid = threadIdx.x;
    if (tid == 0) s.end = kJoinThreads;
    __syncthreads();
    const int next = b + 1 + tid;
    PartInfo other;
    other.req = -1;
    if (next < blocks) other = ws.info[2 * next];
    if (other.req >= 0 && other.last) atomicMin(&s.end, tid);
    __syncthreads();
    const bool mine = other.req >= 0 && tid <= s.end;
    const unsigned votes = __ballot_sync(0xffffffffu, mine);
    if (tid % 32 == 0) s.base[tid / 32] = __popc(votes);
    __syncthreads();
    int at = 1 + __popc(votes & ((1u << tid % 32) - 1u)), parts = 1;
    for (int w = 0; w < kJoinThreads / 32; ++w) {
        at += w < tid / 32 ? s.base[w] : 0;
        parts += s.base[w];
    }
    if (mine) s.slot[at] = 2 * next;
    if (tid == 0) s.slot[0] = 2 * b + 1;
    __syncthreads();
    for (int x = tid; x < parts * kRows; x += kJoinThreads) {
        const float* ml = ws.ml + (size_t)s.slot[x / kRows] * 2 * kTileRows + row0 + x % kRows;
        s.m[x / kRows][x % kRows] = ml[0];
        s.l[x / kRows][x % kRows] = ml[kTileRows];
    }
    __syncthreads();
    return parts;
}

// Joins rows 16 slice .. 16 slice + 15 of a large tile; the parts are added in
// order, so the sum does not depend on which finished first.  A tile's rows
// come in halves of kBigHalf, of which the first `used` hold packed rows.
template <int D, bool kHalf>
__device__ __forceinline__ void join_big(const AttnParams& p, const Workspace& ws, int blocks, int b, int slice,
                                         int used, JoinShared& s)
{
    const PartInfo info = ws.info[2 * b + 1];
    if (info.req < 0) return;
    const int parts = list_parts<kBigTile, 16>(ws, blocks, b, 16 * slice, s);
    constexpr int kPer = 16 * D / kJoinThreads;
    // as the parts lie: rows are neighbours
    const int tid = threadIdx.x, lane_row = tid % 16, row = slice * 16 + lane_row, col = tid / 16 * kPer;
    const Request r = load_request(p, info.req);
    const int packed = info.row0 + row / kBigHalf * used + row % kBigHalf;
    if (row % kBigHalf >= used || packed >= r.q * p.group) return;
    float m = -INFINITY, l = 0.f, out[kPer];
    for (int x = 0; x < parts; ++x) m = max_nan(m, s.m[x][lane_row]);
#pragma unroll
    for (int c = 0; c < kPer; ++c) out[c] = 0.f;
    if (m != -INFINITY) {
#pragma unroll 4
        for (int x = 0; x < parts; ++x) {
            const float w = ex2_approx(s.m[x][lane_row] - m);
            l += w * s.l[x][lane_row];
#pragma unroll
            for (int c = 0; c < kPer; c += 4) {
                const float4 v = *part_columns<kBigTile>(ws, s.slot[x], D, row, col + c);
                out[c] += w * v.x;
                out[c + 1] += w * v.y;
                out[c + 2] += w * v.z;
                out[c + 3] += w * v.w;
            }
        }
    }
    store_row<kPer, kHalf>(p, r, info.kvh, packed, col, out, m, l, kBigShift<kHalf>);
}

// Joins rows 4 slice .. 4 slice + 3 of a small tile.  One long context is a few
// tiles of many parts, and what bounds it is a chain of reads: groups of
// threads, one float4 to a thread, take the parts in turn, and their sums are
// added in order.  (8K keys, 28 heads over 4, the whole call: 27.7 us with a
// block to a tile, 23.7 so.)
template <int D, bool kHalf>
__device__ __forceinline__ void join_small(const AttnParams& p, const Workspace& ws, int blocks, int b, int slice,
                                           JoinShared& s)
{
    constexpr int kRows = kRowsTile / kRowsSlices, kThreads = kRows * D / 4, kGroups = kJoinThreads / kThreads;
    const PartInfo info = ws.info[2 * b + 1];
    if (info.req < 0) return;
    const int parts = list_parts<kRowsTile, kRows>(ws, blocks, b, kRows * slice, s);
    const int group = threadIdx.x / kThreads, t = threadIdx.x % kThreads;
    // as the parts lie: columns are neighbours
    const int lane_row = t / (D / 4), row = slice * kRows + lane_row, col = t % (D / 4) * 4;
    float m = -INFINITY, l = 0.f, out[4] = {0.f, 0.f, 0.f, 0.f};
    for (int x = 0; x < parts; ++x) m = max_nan(m, s.m[x][lane_row]);
    if (m != -INFINITY) {
#pragma unroll 4
        for (int x = group; x < parts; x += kGroups) {
            const float w = ex2_approx(s.m[x][lane_row] - m);
            l += w * s.l[x][lane_row];
            const float4 v = *part_columns<kRowsTile>(ws, s.slot[x], D, row, col);
            out[0] += w * v.x;
            out[1] += w * v.y;
            out[2] += w * v.z;
            out[3] += w * v.w;
        }
    }
    __syncthreads();    // m and l are free
    float4* sum = reinterpret_cast<float4*>(s.m);
    float* total = s.l[0];
    sum[threadIdx.x] = make_float4(out[0], out[1], out[2], out[3]);
    total[threadIdx.x] = l;
    __syncthreads();
    const Request r = load_request(p, info.req);
    const int packed = info.row0 + row;
    if (group > 0 || packed >= r.q * p.group) return;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) {
        const float4 v = sum[g * kThreads + t];
        l += total[g * kThreads + t];
        out[0] += v.x;
        out[1] += v.y;
        out[2] += v.z;
        out[3] += v.w;
    }
    store_row<4, kHalf>(p, r, info.kvh, packed, col, out, m, l, Operand<kHalf>::kShift);
}

// Slices 0 .. kBigSlices - 1 of the large tiles, then those of the small ones.
// Five blocks to an SM leave the registers that four parts in flight take: with
// eight (the compiler's choice) 10 contexts of up to 69K, 12 heads on one, take
// 58 us instead of 53, with three 509 tokens over 4K 54 instead of 52.
template <int D, bool kHalf>
__global__ void __launch_bounds__(kJoinThreads, 5)
paged_join_kernel(const AttnParams p, const Workspace rows, const Workspace big, int blocks, int used, int first_slice)
{
    __shared__ JoinShared s;
    wait_for_previous();
    const int slice = blockIdx.y + first_slice;
    if (slice >= kBigSlices) join_small<D, kHalf>(p, rows, blocks, blockIdx.x, slice - kBigSlices, s);
    else join_big<D, kHalf>(p, big, blocks, blockIdx.x, slice, used, s);
}

}  // namespace paged
}  // namespace ra
