// paged_tiles.cuh -- attention of many new tokens over a paged cache, on the
// tensor cores: the form of paged_attn_fwd for prompt chunks.
//
// A block holds two tiles of 128 packed rows (token, head of the group) of
// one request and key/value head; both share every tile of 128 keys.
//   warp 0      copies Q once and K/V tiles page by page (TMA; a page's rows
//               are boxes of a 4-D tensor map, one lane issues one box)
//   warp 1      tensor memory and the MMAs: S = Q K^T, O += P V
//   warps 2-3   look through V, a half of each tile each, where some row does
//               not see some key (see below)
//   warps 4-7   softmax and results of tile 0
//   warps 8-11  the same of tile 1
// Tensor memory (512 columns): S0, S1 of 128 columns, then O0, O1.  P, rounded
// to the operand type (off by 2^-8 or 2^-11 of itself at most; the row sums take it
// unrounded), overwrites the first 64 columns of its S, so the next S comes
// behind P V.  With d 64 there is room for P of its own, and the next S is
// computed while the softmax of this one runs: 1.49 -> 1.43 us a key tile.
// (Two S of 64 keys instead, which d 128 has room for, are slower: 2.90 us a key
// tile against 1.73, as the hand-offs between the warps double.  Key tiles in
// turn to both softmax groups where there is one row tile only, and rows stored
// through shared memory, gave nothing.)
//
// The work is cut into equal, contiguous shares of (request, key/value head,
// tile, key tile), one for each SM: with as few tiles as a single chunk of a
// few hundred tokens has, whole tiles would leave most SMs idle.  Every role
// walks its block's share by itself, from the same start.
//
// Bound, at d 128, by the softmax and its tile's two products taking turns (of
// 2650 cycles a key tile, 1400 and 1250; the tensor core is at work for 2050 of
// them), at d 64 by latency: an instruction in 46 % of the cycles, exponentials
// 40 %, tensor cores 39 %; in the other cycles no warp is ready, as two softmax
// warps to a scheduler do not hide their own chains.  2048 tokens at the end of
// 64K, 32 heads over 8: 1.53 us a key tile, 1670 TFLOP/s (0.86 of measured) at d
// 128, 1.30 us at d 64, calls apart.  Back to back, when power lowers the clock,
// 2048 over 128K run at 1540 TFLOP/s.  Short pieces cost 5 to 6 us beside their
// keys (kExtra).
// Blocks of one key/value head read its keys at the same time, from L2 (see
// Walk::key_tile).
#pragma once

#include <new>

#include "paged_attn.cuh"

namespace ra {
namespace paged {
namespace tiles {

constexpr int kBM = kBigHalf;      // packed rows of a tile
constexpr int kBN = 128;           // keys of a key tile
constexpr int kTiles = 2;          // row tiles of a block
constexpr int kTileRows = kTiles * kBM;
static_assert(kTileRows == kBigTile, "parts are joined as they are cut");
constexpr int kThreads = 384;
// Registers of warps 0-3 and of warps 4-11: 128 * 104 + 256 * 200 are the 384 *
// 168 that the block starts with.
constexpr int kFewRegs = 104, kManyRegs = 200;
constexpr float kRescaleThreshold = 8.0f;   // log2 units

template <int D>
struct Cfg {
    static constexpr int kBoxes = D / 64;                       // 64-column boxes of a tile
    static constexpr int kBoxBytes = 64 * kBN * 2;
    static constexpr int kTileBytes = kBN * D * 2;
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kTiles * kTileBytes;
    static constexpr int kOffV = kOffK + kStages * kTileBytes;
    static constexpr int kOffBar = kOffV + kStages * kTileBytes;
    static constexpr int kBarBytes = 512;
    static constexpr int kSmemBytes = kOffBar + kBarBytes + 1024;   // + alignment slack
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kColS = 0;          // S_u at kColS + 128 u
    static constexpr uint32_t kColO = 256;        // O_u at kColO + D u
    static constexpr bool kOwnP = D == 64;
    static constexpr uint32_t kColP = kOwnP ? kColO + 2 * D : kColS;      // P_u at kColP + kPitchP u
    static constexpr uint32_t kPitchP = kOwnP ? 64 : 128;
};

// The weights' reference (see Operand): the running maximum may lag by up to
// 2^8, so fp16 weights stay below 2^15.
template <bool kHalf> constexpr float kShift = kBigShift<kHalf>;

struct TileParams {
    AttnParams a;
    Workspace ws;
    RowRange range;
    int tok_tile;           // tokens of a row tile: 128 / group, rounded down
    int box_rows;           // rows of a K/V box: the largest power of two in page_size, at most 128
    uint64_t wait_limit_ns;
};

// What a tile costs beside its key tiles, in key tiles: Q has to arrive, the
// pipeline to fill and to drain, and the results to be written, 5 to 6 us
// against 1.3 to 1.6 us for a key tile.  40 requests with 5 chunks of up to 1024
// tokens, d 64: 319 us without it, 254 with 2, 241 with 3 or 4, 254 with 6.
constexpr int kExtra = 3;

// The least share of a block, in key tiles: a little work on few blocks has
// fewer parts to write and to join (17 tokens over 19K, 12 heads on one: 66 us
// without it, 42 with 5 or 8; 509 tokens on their own: 36, 38 and 43 us).
constexpr int kMinShare = 5;

// A block's place in its share: key tiles [k0, k1) of a tile, of `total`.
struct Walk {
    const TileParams& p;
    Request r;
    TileWork w;
    int req, kvh, t, k0, k1, total;
    int turn;                // see key_tile
    unsigned passed;         // key tiles of the pieces so far
    long long left;          // cost of what follows this piece

    __device__ __forceinline__ Walk(const TileParams& p_, int req_, int kvh_, int t_, long long c0, long long share)
        : p(p_), req(req_), kvh(kvh_), t(t_), passed(0u), left(share)
    {
        load();
        cut(c0);
    }
    static __device__ __forceinline__ TileWork work(const TileParams& p, const Request& r)
    {
        return TileWork{r.q, r.len, p.a.causal, kTiles * p.tok_tile, kBN, kExtra};
    }
    static __device__ __forceinline__ long long cost(const TileParams& p, int i)
    {
        const Request r = load_request(p.a, i);
        if (!p.range.has(r.q * p.a.group)) return 0;
        const TileWork w = work(p, r);
        return w.before(w.tiles()) * p.a.kv_heads;
    }
    __device__ __forceinline__ void load()
    {
        r = load_request(p.a, req);
        w = work(p, r);
    }
    // The piece that begins at cost c0 of the tile.
    __device__ __forceinline__ void cut(long long c0)
    {
        total = w.units(t);
        const long long c1 = min((long long)total + kExtra, c0 + left);
        left -= c1 - c0;
        k0 = cut_units(c0, kExtra);
        k1 = cut_units(c1, kExtra);
        turn = k1 - k0 == total ? (int)(passed % (unsigned)total) : 0;
        passed += (unsigned)(k1 - k0);
    }
    // The j-th key tile of the piece: from the last to the first, so that the
    // blocks that take over a tile of the same keys, which all begin at its end,
    // read them at the same time, and those that leave one to the next block,
    // which all end at its beginning, too.  A whole tile between the two goes
    // round from where the pieces before it got to.  L2 then serves what HBM had
    // to: 2048 tokens over 128K, calls apart, 2936 us in ascending order, 2846 descending,
    // 2624 with whole tiles turned.
    __device__ __forceinline__ int key_tile(int j) const
    {
        const int kt = k1 - 1 - j - turn;
        return kt < k0 ? kt + (k1 - k0) : kt;
    }
    // The share ends in front of the tile's first key tile.
    __device__ __forceinline__ bool empty() const { return k0 == k1; }
    __device__ __forceinline__ int tok0() const { return t * w.step; }
    // first key tile of this piece with a key that the block's first row does
    // not see, or k1
    __device__ __forceinline__ int first_masked() const
    {
        const int last = p.a.causal ? r.len - r.q + tok0() : r.len - 1;
        return min(k1, max(k0, last < 0 ? 0 : (last + 1) / kBN));
    }
    // row tiles that hold tokens
    __device__ __forceinline__ int row_tiles() const { return r.q - tok0() > p.tok_tile ? 2 : 1; }
    // To the next piece of work; false behind the last one.
    __device__ __forceinline__ bool next()
    {
        if (left == 0) return false;
        if (++t == w.tiles()) {
            t = 0;
            if (++kvh == p.a.kv_heads) {
                kvh = 0;
                do {
                    ++req;
                    load();
                } while (!p.range.has(r.q * p.a.group));    // some later request has the work that is left
            }
        }
        cut(0);
        return !empty();
    }
};

__device__ __forceinline__ uint32_t bits_of(uint32_t packed, int odd) { return odd ? packed >> 16 : packed & 0xffffu; }
template <bool kHalf> __device__ __forceinline__ float widen(uint32_t bits)
{
    if constexpr (kHalf) return __half2float(__ushort_as_half((unsigned short)bits));
    else return __uint_as_float(bits << 16);
}

// O += P V of one or both halves of a key tile for the rows of one warp, key by
// key and only for the keys that a row sees.  `init`: O holds nothing yet.
template <int D, bool kHalf>
__device__ __forceinline__ void add_seen_keys(const AttnParams& a, const int* table, int kvh, int key0, int valid, int lim,
                                              bool lower, bool upper, uint32_t tS, uint32_t tO, bool init)
{
#pragma unroll 1
    for (int half = lower ? 0 : 1; half < (upper ? 2 : 1); ++half) {
        uint32_t pk[32];
        tmem_ld32(tS + 32u * half, pk);
        tmem_ld_wait(pk);
        uint32_t weight[32];     // indexed at run time: lives in local memory
        for (int c = 0; c < 32; ++c) weight[c] = pk[c];
#pragma unroll 1
        for (int c4 = 0; c4 < D / 32; ++c4) {
            uint32_t o[32];
            if (!init || (half == 1 && lower)) {
                tmem_ld32(tO + 32u * c4, o);
                tmem_ld_wait(o);
            } else {
#pragma unroll
                for (int c = 0; c < 32; ++c) o[c] = 0u;
            }
#pragma unroll 1
            for (int k = 0; k < 64 && 64 * half + k < valid; ++k) {
                const int key = key0 + 64 * half + k;
                const int pi = page_index(key, a.page_size, a.page_shift), page = table[pi];
                if (!page_ok(page, a.num_pages)) continue;
                const uint4* row = reinterpret_cast<const uint4*>(
                    a.vc + row_offset(a.lv, page, key - pi * a.page_size, kvh) + 32 * c4);
                if (key > lim) continue;
                const float wgt = widen<kHalf>(bits_of(weight[k >> 1], k & 1));
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const uint4 x = row[v];
                    const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int z = 0; z < 8; ++z)
                        o[8 * v + z] = __float_as_uint(fmaf(wgt, widen<kHalf>(bits_of(y[z >> 1], z & 1)),
                                                            __uint_as_float(o[8 * v + z])));
                }
            }
            __syncwarp();
            tmem_st32(tO + 32u * c4, o);
            tmem_st_wait();
        }
    }
}

template <int D, bool kHalf>
__global__ void __launch_bounds__(kThreads, 1)
paged_tiles_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const __grid_constant__ TileParams p)
{
    using CF = Cfg<D>;
    using Op = Operand<kHalf>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ long long s_scratch[kThreads / 32 + 1];
    __shared__ int s_start[3];             // request, key/value head, tile
    __shared__ long long s_offset, s_cost; // cost in front of the share, into the request and the tile
    __shared__ int s_seen[2];              // piece whose O tile u holds sums before its first MMA
    __shared__ int s_odd[CF::kStages][2];  // key tile whose V half holds an infinity or a NaN
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw_base);
    const uint32_t sQ = base + CF::kOffQ, sK = base + CF::kOffK, sV = base + CF::kOffV;
    const uint32_t bar0 = base + CF::kOffBar;
    const uint32_t bar_q_full = bar0, bar_q_empty = bar0 + 8u;
    auto bar_k_full = [&](int s) { return bar0 + 8u * (2 + s); };
    auto bar_k_empty = [&](int s) { return bar0 + 8u * (2 + CF::kStages + s); };
    auto bar_v_full = [&](int s) { return bar0 + 8u * (2 + 2 * CF::kStages + s); };
    auto bar_v_empty = [&](int s) { return bar0 + 8u * (2 + 3 * CF::kStages + s); };
    const uint32_t bar_misc = bar0 + 8u * (2 + 4 * CF::kStages);
    auto bar_s_full = [&](int u) { return bar_misc + 8u * u; };          // MMA -> softmax
    auto bar_p_full = [&](int u) { return bar_misc + 8u * (2 + u); };    // softmax -> MMA
    auto bar_o = [&](int u) { return bar_misc + 8u * (4 + u); };         // P V done: each (own P), or a piece's last
    auto bar_s_taken = [&](int u) { return bar_misc + 8u * (6 + u); };   // softmax -> MMA: S read (own P)
    const uint32_t bar_drain = bar_misc + 8u * 8;
    auto bar_check = [&](int s) { return bar_misc + 8u * (9 + s); };     // V looked through
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + CF::kOffBar + 448);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + CF::kOffBar + 456);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const AttnParams& a = p.a;
    let_next_start();

    // ---- this block's share of the work
    const int G = gridDim.x, b = blockIdx.x;
    const int per = (a.n + kThreads - 1) / kThreads;
    const int i0 = min(a.n, tid * per), i1 = min(a.n, i0 + per);
    long long mine = 0, total;
    for (int i = i0; i < i1; ++i) mine += Walk::cost(p, i);
    const long long before = block_exclusive_sum(mine, s_scratch, &total);
    const int sharing = total >= (long long)G * kMinShare ? G : max(1, (int)total / kMinShare);
    Share share{0, 0};
    if (b < sharing) share = share_of(total, sharing, b);
    const long long start = share.start;
    if (tid < 2) p.ws.info[2 * b + tid].req = -1;
    if (share.count == 0) {
        wait_for_previous();
        return;
    }

    WaitCtl wc{abort_flag, a.status, p.wait_limit_ns};
    if (tid == 0) {
        *abort_flag = 0;
        mbar_init(bar_q_full, 1);
        mbar_init(bar_q_empty, 1);
        for (int s = 0; s < CF::kStages; ++s) {
            mbar_init(bar_k_full(s), 1);
            mbar_init(bar_k_empty(s), 1);
            mbar_init(bar_v_full(s), 1);
            mbar_init(bar_v_empty(s), 3);      // P V and both checking warps
            mbar_init(bar_check(s), 2);
            s_odd[s][0] = s_odd[s][1] = 0;
        }
        for (int u = 0; u < kTiles; ++u) {
            mbar_init(bar_s_full(u), 1);
            mbar_init(bar_p_full(u), kBM);
            mbar_init(bar_o(u), 1);
            mbar_init(bar_s_taken(u), kBM);
            s_seen[u] = 0;
        }
        mbar_init(bar_drain, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), CF::kTmemCols);
        tmem_relinquish();
    }
    if (before <= start && start < before + mine) {
        long long x = start - before;
        int i = i0;
        for (long long c; x >= (c = Walk::cost(p, i)); ++i) x -= c;
        s_start[0] = i;
        s_offset = x;
    }
    __syncthreads();
    {
        // the tile: every thread knows the cost before one of kThreads of them
        const TileWork w = Walk::work(p, load_request(a, s_start[0]));
        const int count = w.tiles(), each = (count + kThreads - 1) / kThreads;
        const int lo = min(count, tid * each), hi = min(count, lo + each);
        const long long head = w.before(count);
        const int kvh = quotient_below(s_offset, head, a.kv_heads);
        const long long x = s_offset - kvh * head;
        if (lo < hi && w.before(lo) <= x && x < w.before(hi)) {
            const int t = w.tile_of(x, lo, hi);
            s_start[1] = kvh;
            s_start[2] = t;
            s_cost = x - w.before(t);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Walk walk(p, s_start[0], s_start[1], s_start[2], s_cost, share.count);
    const bool any = !walk.empty();
    // The softmax warps keep theirs in shared memory: with 128 scores in
    // registers there is no room for it beside them.
    __shared__ __align__(16) uint8_t s_walk[8][sizeof(Walk)];

    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == 0) {
        // ------------------------------------------------------------ copies
        const int boxes = kBN / p.box_rows * CF::kBoxes;     // at most 32: one for each lane
        const int box = lane / CF::kBoxes, half = lane % CF::kBoxes;
        const uint32_t box_dst = (uint32_t)(half * CF::kBoxBytes + box * p.box_rows * 128);
        const uint32_t q_bytes = (uint32_t)(p.tok_tile * a.group * 128 * CF::kBoxes);
        if (lane == 0) {
            tma_prefetch_desc(&map_q);
            tma_prefetch_desc(&map_k);
            tma_prefetch_desc(&map_v);
        }
        int last_k[CF::kStages], last_v[CF::kStages], last_q = -1;   // parity of the last copy issued
        for (int s = 0; s < CF::kStages; ++s) last_k[s] = last_v[s] = -1;
        auto wait_all = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait_inline(bar, parity, wc));
        };
        bool ok = true;
        uint32_t n = 0, piece = 0;
        if (any) do {
            const int* table = a.table + (long long)walk.req * a.table_stride;
            const int keys = walk.w.keys(walk.t), count = walk.k1 - walk.k0, nu = walk.row_tiles();
            auto page_at = [&](int j) {
                const int key = walk.key_tile(j) * kBN + box * p.box_rows;
                return lane < boxes && j < count && key < keys
                           ? table[page_index(key, a.page_size, a.page_shift)] : 0;
            };
            int page = page_at(0);
            if (!(ok = wait_all(bar_q_empty, (piece & 1u) ^ 1u))) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar_q_full, q_bytes * nu);
                for (int u = 0; u < nu; ++u)
                    for (int x = 0; x < CF::kBoxes; ++x)
                        tma_load_4d(sQ + u * CF::kTileBytes + x * CF::kBoxBytes, &map_q, bar_q_full, 64 * x, 0,
                                    walk.r.first + walk.tok0() + u * p.tok_tile, walk.kvh);
            }
            last_q = (int)(piece & 1u);
            for (int j = 0; j < count; ++j, ++n) {
                const int s = n % CF::kStages;
                const uint32_t ph = (n / CF::kStages) & 1u;
                const int key = walk.key_tile(j) * kBN + box * p.box_rows;
                const bool load = lane < boxes && key < keys;
                // a page outside the pool: a coordinate outside the map, which reads as zeros
                int coord = page;
                if (load && !page_ok(page, a.num_pages)) {
                    coord = a.num_pages;
                    atomicOr(a.status, kStatusBadPage);
                }
                const int off = key - page_index(key, a.page_size, a.page_shift) * a.page_size;
                page = page_at(j + 1);
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, load)) * p.box_rows * 128u;
                if (!(ok = wait_all(bar_k_empty(s), ph ^ 1u))) break;
                if (lane == 0) mbar_arrive_expect_tx(bar_k_full(s), bytes);
                __syncwarp();
                if (load)
                    tma_load_4d(sK + s * CF::kTileBytes + box_dst, &map_k, bar_k_full(s), 64 * half, off, walk.kvh, coord);
                last_k[s] = (int)ph;
                if (!(ok = wait_all(bar_v_empty(s), ph ^ 1u))) break;
                if (lane == 0) mbar_arrive_expect_tx(bar_v_full(s), bytes);
                __syncwarp();
                if (load)
                    tma_load_4d(sV + s * CF::kTileBytes + box_dst, &map_v, bar_v_full(s), 64 * half, off, walk.kvh, coord);
                last_v[s] = (int)ph;
            }
            ++piece;
        } while (ok && walk.next());
        if (!ok) {
            // Let every copy still in flight land before the block exits.
            volatile int dummy = 0;
            WaitCtl drain{&dummy, a.status, 200000000ull};
            if (last_q >= 0) mbar_wait_inline(bar_q_full, (uint32_t)last_q, drain);
            for (int s = 0; s < CF::kStages; ++s) {
                if (last_k[s] >= 0) mbar_wait_inline(bar_k_full(s), (uint32_t)last_k[s], drain);
                if (last_v[s] >= 0) mbar_wait_inline(bar_v_full(s), (uint32_t)last_v[s], drain);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // -------------------------------------------------------------- MMA
        // The whole warp runs converged; one elected lane issues the MMAs and
        // commits.  MMAs run in the order of issue, so the next S = Q K^T,
        // issued after P V, does not overwrite P early.
        constexpr uint32_t kType = kHalf ? 0u : (1u << 7) | (1u << 10);
        constexpr uint32_t kTypeMask = ~((1u << 7) | (1u << 10));
        constexpr uint32_t idesc_qk = (idesc_bf16_f32(kBM, kBN, false, false) & kTypeMask) | kType;
        constexpr uint32_t idesc_pv = (idesc_bf16_f32(kBM, D, false, true) & kTypeMask) | kType;
        const uint64_t dq0 = sdesc_sw128(sQ, 16, 1024);
        const uint64_t dk0 = sdesc_sw128(sK, 16, 1024);
        const uint64_t dv0 = sdesc_sw128(sV, CF::kBoxBytes, 1024);
        constexpr uint32_t kTile16 = CF::kTileBytes >> 4, kBox16 = CF::kBoxBytes >> 4;
        auto issue_s = [&](int u, int s) {
            const uint64_t dq = dq0 + (uint32_t)u * kTile16, dk = dk0 + (uint32_t)s * kTile16;
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off16 = (kk >> 2) * kBox16 + (kk & 3) * 2;
                    mma_bf16_ss(tmem + CF::kColS + 128u * u, dq + off16, dk + off16, idesc_qk, kk > 0 ? 1u : 0u);
                }
            }
            __syncwarp();
        };
        auto issue_pv = [&](int u, int s, bool first) {
            const uint64_t dv = dv0 + (uint32_t)s * kTile16;
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kBN / 16; ++kk)
                    mma_bf16_ts(tmem + CF::kColO + (uint32_t)D * u, tmem + CF::kColP + CF::kPitchP * u + 8u * kk,
                                dv + (uint32_t)kk * (2048 >> 4), idesc_pv, (first && kk == 0) ? 0u : 1u);
            }
            __syncwarp();
        };
        auto commit = [&](uint32_t bar) {
            if (elect_one()) mma_commit(bar);
            __syncwarp();
        };
        auto wait_all = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait_inline(bar, parity, wc));
        };
        bool ok = true;
        uint32_t n = 0, piece = 0, done[2] = {0, 0};      // key tiles; pieces; weights of tile u taken
        if constexpr (CF::kOwnP) {
            // S of the next key tile as soon as both softmax groups have read
            // this one's, then P V of this one.
            uint32_t issued[2] = {0, 0};                  // S of tile u
            auto next_s = [&](int nu, int s) {
                for (int u = 0; u < nu; ++u) {
                    if (issued[u] > 0 && !wait_all(bar_s_taken(u), (issued[u] - 1) & 1u)) return false;
                    ++issued[u];
                    tc_fence_after();
                    issue_s(u, s);
                    commit(bar_s_full(u));
                }
                commit(bar_k_empty(s));
                return true;
            };
            if (any) do {
                const int count = walk.k1 - walk.k0, nu = walk.row_tiles();
                const int s0 = n % CF::kStages;
                if (!(ok = wait_all(bar_q_full, piece & 1u) && wait_all(bar_k_full(s0), (n / CF::kStages) & 1u))) break;
                tc_fence_after();
                if (!(ok = next_s(nu, s0))) break;
                if (count == 1) commit(bar_q_empty);
                for (int j = 0; j < count && ok; ++j, ++n) {
                    const int s = n % CF::kStages, s1 = (n + 1) % CF::kStages;
                    if (j + 1 < count) {
                        if (!(ok = wait_all(bar_k_full(s1), ((n + 1) / CF::kStages) & 1u) && next_s(nu, s1))) break;
                        if (j + 2 == count) commit(bar_q_empty);
                    }
                    if (!(ok = wait_all(bar_v_full(s), (n / CF::kStages) & 1u))) break;
                    for (int u = 0; u < nu; ++u) {
                        if (!(ok = wait_all(bar_p_full(u), done[u] & 1u))) break;
                        ++done[u];
                        tc_fence_after();
                        issue_pv(u, s, j == 0 && *(volatile int*)&s_seen[u] != (int)(piece + 1));
                        commit(bar_o(u));
                    }
                    if (ok) commit(bar_v_empty(s));
                }
                ++piece;
            } while (ok && walk.next());
        } else
        if (any) do {
            const int count = walk.k1 - walk.k0, nu = walk.row_tiles();
            const int s0 = n % CF::kStages;
            if (!(ok = wait_all(bar_q_full, piece & 1u) && wait_all(bar_k_full(s0), (n / CF::kStages) & 1u))) break;
            tc_fence_after();
            for (int u = 0; u < nu; ++u) {
                issue_s(u, s0);
                commit(bar_s_full(u));
            }
            commit(bar_k_empty(s0));
            if (count == 1) commit(bar_q_empty);
            for (int j = 0; j < count && ok; ++j, ++n) {
                const int s = n % CF::kStages, s1 = (n + 1) % CF::kStages;
                const bool more = j + 1 < count;
                if (!(ok = wait_all(bar_v_full(s), (n / CF::kStages) & 1u))) break;
                for (int u = 0; u < nu; ++u) {
                    if (!(ok = wait_all(bar_p_full(u), done[u] & 1u))) break;
                    ++done[u];
                    tc_fence_after();
                    const bool first = j == 0 && *(volatile int*)&s_seen[u] != (int)(piece + 1);
                    issue_pv(u, s, first);
                    if (!more) commit(bar_o(u));
                    if (u == nu - 1) commit(bar_v_empty(s));
                    if (more) {
                        if (u == 0) {
                            if (!(ok = wait_all(bar_k_full(s1), ((n + 1) / CF::kStages) & 1u))) break;
                            tc_fence_after();
                        }
                        issue_s(u, s1);
                        commit(bar_s_full(u));
                        if (u == nu - 1) {
                            commit(bar_k_empty(s1));
                            if (j + 2 == count) commit(bar_q_empty);
                        }
                    }
                }
            }
            ++piece;
        } while (ok && walk.next());
        // Every MMA issued so far must finish before tensor memory is released.
        commit(bar_drain);
        volatile int dummy = 0;
        WaitCtl drain{&dummy, a.status, 200000000ull};
        __all_sync(0xffffffffu, mbar_wait_inline(bar_drain, 0, drain));
    } else {
        // ------------------------------------------------------------ checks
        // In a key tile with a key that some row does not see, a weight of 0
        // does not hide an infinity or a NaN in V.  Rows of V behind the last
        // key in use, which may never have been written, are cleared; and if a
        // row in use holds one, this warp's half of V is cleared and the
        // softmax warps add its keys one by one to the rows that see them.
        // They see every key tile and hold its V until then, so bar_v_full is
        // never a phase ahead of them, nor they of it.
        const int half = warp - 2;
        bool ok = true;
        uint32_t n = 0;
        if (any) do {
            const int count = walk.k1 - walk.k0, keys = walk.w.keys(walk.t), masked = walk.first_masked();
            for (int j = 0; j < count; ++j, ++n) {
                const int kt = walk.key_tile(j), s = n % CF::kStages, valid = keys - kt * kBN;
                ok = __all_sync(0xffffffffu, mbar_wait_inline(bar_v_full(s), (n / CF::kStages) & 1u, wc));
                if (!ok) break;
                if (kt < masked) {
                    if (lane == 0) mbar_arrive(bar_v_empty(s));
                    continue;
                }
                uint4* v = reinterpret_cast<uint4*>(gbase + CF::kOffV + s * CF::kTileBytes);
                // a box's rows are 8 pieces of 16 bytes; four rows to a pass
                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                bool odd = false;
                for (int x = 0; x < CF::kBoxes; ++x) {
                    uint4* at = v + (x * kBN + half * 64) * 8 + lane;
#pragma unroll 4
                    for (int y = 0; y < 16; ++y) {
                        if (half * 64 + 4 * y + (lane >> 3) < valid) {
                            const uint4 z = at[32 * y];
                            odd |= Op::nonfinite(z.x) || Op::nonfinite(z.y) || Op::nonfinite(z.z) || Op::nonfinite(z.w);
                        } else {
                            at[32 * y] = zero;
                        }
                    }
                }
                if (__any_sync(0xffffffffu, odd)) {
                    for (int x = 0; x < CF::kBoxes; ++x)
                        for (int y = 0; y < 16; ++y) v[(x * kBN + half * 64) * 8 + lane + 32 * y] = zero;
                    *(volatile int*)&s_odd[s][half] = (int)(n + 1);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar_check(s));
                    mbar_arrive(bar_v_empty(s));
                }
            }
        } while (ok && walk.next());
    }
    } else {
        // ------------------------------------------------- softmax + results
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        const int u = (warp - 4) >> 2;                 // row tile
        const uint32_t quarter = (uint32_t)(warp & 3); // tensor memory lane quarter
        const int row = (int)quarter * 32 + lane;
        const uint32_t tS = tmem_addr(tmem, quarter * 32, CF::kColS + 128u * u);
        const uint32_t tP = tmem_addr(tmem, quarter * 32, CF::kColP + CF::kPitchP * u);
        const uint32_t tO = tmem_addr(tmem, quarter * 32, CF::kColO + (uint32_t)D * u);
        const float sl2 = a.scale_log2;
        const int used = p.tok_tile * a.group;
        Walk* const place = reinterpret_cast<Walk*>(s_walk[warp - 4]);
        if (lane == 0) new (place) Walk(walk);
        __syncwarp();
        bool ok = true, more = any;
        uint32_t n = 0, piece = 0, seen = 0, outs = 0, looked = 0;    // looked: parities of bar_check
        while (ok && more) {
            const Walk& walk = *place;
            const int count = walk.k1 - walk.k0, nu = walk.row_tiles(), masked = walk.first_masked();
            const int packed = walk.tok0() * a.group + u * used + row;
            const int tok = packed / a.group;
            const bool store = row < used && tok < walk.r.q;
            // last key that the row and the tile's first row see
            const int past = walk.r.len - walk.r.q;
            const int lim = a.causal ? past + min(tok, walk.r.q - 1) : walk.r.len - 1;
            const int lim_tile = a.causal ? past + walk.tok0() + u * p.tok_tile : walk.r.len - 1;
            float m_used = -INFINITY;   // reference of the exponentials (log2), without the shift
            float l = 0.f;
            if (u < nu) {
                for (int j = 0; j < count; ++j, ++n, ++seen) {
                    // all lanes leave together: the tcgen05 loads below are warp-wide
                    ok = __all_sync(0xffffffffu, mbar_wait_inline(bar_s_full(u), seen & 1u, wc));
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t s[128];
#pragma unroll
                    for (int c4 = 0; c4 < 4; ++c4)
                        tmem_ld32(tS + 32u * c4, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * c4]));
                    tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(&s[0]));
                    tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(&s[32]));
                    tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(&s[64]));
                    tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(&s[96]));
                    if constexpr (CF::kOwnP) {
                        tc_fence_before();
                        mbar_arrive(bar_s_taken(u));
                    }
                    const int key0 = walk.key_tile(j) * kBN;
                    if (key0 + kBN - 1 > lim_tile) {
                        const int last = lim - key0;
#pragma unroll
                        for (int c = 0; c < 128; ++c)
                            if (c > last) s[c] = __float_as_uint(-INFINITY);
                    }
                    // Row maximum: four independent chains of 3-input maxima.
                    float mq[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) mq[x] = __uint_as_float(s[x]);
#pragma unroll
                    for (int c = 4; c < 124; c += 8) {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            mq[x] = max3f(mq[x], __uint_as_float(s[c + 2 * x]), __uint_as_float(s[c + 2 * x + 1]));
                    }
                    mq[0] = max3f(mq[0], __uint_as_float(s[124]), __uint_as_float(s[125]));
                    mq[1] = max3f(mq[1], __uint_as_float(s[126]), __uint_as_float(s[127]));
                    const float m_new = max3f(mq[0], mq[1], fmaxf(mq[2], mq[3])) * sl2;
                    // The reference is raised only when the maximum is above
                    // it by more than 2^8; O and l share it, so results are exact.
                    const bool raise = m_new > m_used + kRescaleThreshold;
                    float alpha = 1.f;
                    if (raise) {
                        alpha = ex2_approx(m_used - m_new);   // 0 when m_used = -inf
                        m_used = m_new;
                    }
                    const float mb = m_used == -INFINITY ? 0.f : m_used - kShift<kHalf>;
                    float sp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 128; c += 2) {
                        float p0, p1;
                        fma2(p0, p1, __uint_as_float(s[c]), __uint_as_float(s[c + 1]), sl2, sl2, -mb, -mb);
                        p0 = ex2_approx(p0);
                        p1 = ex2_approx(p1);
                        const int x = (c >> 1) & 1;
                        add2(sp[2 * x], sp[2 * x + 1], p0, p1);
                        s[c >> 1] = Op::pack(p0, p1);
                    }
                    if (CF::kOwnP && j > 0) {
                        // the P V before this one has read P, and left O
                        ok = __all_sync(0xffffffffu, mbar_wait_inline(bar_o(u), outs & 1u, wc));
                        if (!ok) break;
                        ++outs;
                        tc_fence_after();
                    }
                    tmem_st32(tP, *reinterpret_cast<const uint32_t(*)[32]>(&s[0]));
                    tmem_st32(tP + 32u, *reinterpret_cast<const uint32_t(*)[32]>(&s[32]));
                    l = l * alpha + ((sp[0] + sp[1]) + (sp[2] + sp[3]));
                    if (j > 0 && __any_sync(0xffffffffu, raise)) {
                        // O_u is idle: without its own P, the S_u just read was issued
                        // after the last P_u V and its end covers every earlier MMA.
#pragma unroll
                        for (int c4 = 0; c4 < D / 32; ++c4) {
                            uint32_t o[32];
                            tmem_ld32(tO + 32u * c4, o);
                            tmem_ld_wait(o);
#pragma unroll
                            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                            tmem_st32(tO + 32u * c4, o);
                        }
                    }
                    tmem_st_wait();
                    if (key0 >= masked * kBN) {
                        // warps 2-3 have looked through V (see there)
                        const int vs = n % CF::kStages;
                        ok = __all_sync(0xffffffffu, mbar_wait_inline(bar_check(vs), looked >> vs & 1u, wc));
                        if (!ok) break;
                        looked ^= 1u << vs;
                        const int mark = (int)(n + 1);
                        const bool lower = *(volatile int*)&s_odd[vs][0] == mark;
                        const bool upper = *(volatile int*)&s_odd[vs][1] == mark;
                        if (lower || upper) {
                            add_seen_keys<D, kHalf>(a, a.table + (long long)walk.req * a.table_stride, walk.kvh, key0,
                                                    min(kBN, walk.w.keys(walk.t) - key0), lim, lower, upper, tP, tO, j == 0);
                            if (j == 0) *(volatile int*)&s_seen[u] = (int)(piece + 1);
                        }
                    }
                    tc_fence_before();
                    mbar_arrive(bar_p_full(u));
                }
            } else {
                for (int j = 0; j < count; ++j, ++n)
                    if (walk.key_tile(j) >= masked) looked ^= 1u << (n % CF::kStages);
            }
            if (ok && u < nu) ok = __all_sync(0xffffffffu, mbar_wait_inline(bar_o(u), outs++ & 1u, wc));
            if (ok && u < nu) {
                tc_fence_after();
                const bool whole = count == walk.total;
                if (whole) {
                    const bool none = m_used == -INFINITY && l == 0.f;    // no key with a weight
                    const float inv = none ? 0.f : 1.f / l;
                    const int head = walk.kvh * a.group + (packed - tok * a.group);
                    uint16_t* dst = a.o + (long long)(walk.r.first + tok) * a.o_tok + (long long)head * a.o_head;
#pragma unroll
                    for (int c4 = 0; c4 < D / 32; ++c4) {
                        uint32_t o[32];
                        tmem_ld32(tO + 32u * c4, o);
                        tmem_ld_wait(o);
                        uint32_t pk[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            pk[c] = Op::pack(__uint_as_float(o[2 * c]) * inv, __uint_as_float(o[2 * c + 1]) * inv);
                        if (store) {
                            uint4* d4 = reinterpret_cast<uint4*>(dst + 32 * c4);
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                d4[x] = make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
                        }
                    }
                    if (store)
                        a.lse[(long long)head * a.tokens + walk.r.first + tok] =
                            none ? -INFINITY : (m_used - kShift<kHalf> + log2f(l)) * 0.69314718055994531f;
                } else {
                    const int slot = 2 * b + (walk.k0 == 0);
#pragma unroll
                    for (int c4 = 0; c4 < D / 32; ++c4) {
                        uint32_t o[32];
                        tmem_ld32(tO + 32u * c4, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            *part_columns<kTileRows>(p.ws, slot, D, u * kBM + row, 32 * c4 + 4 * x) = make_float4(
                                __uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]),
                                __uint_as_float(o[4 * x + 2]), __uint_as_float(o[4 * x + 3]));
                    }
                    // a NaN sum without a maximum (every score NaN) must not read as "no key"
                    float* ml = p.ws.ml + (size_t)slot * 2 * kTileRows + u * kBM + row;
                    ml[0] = l == l ? m_used : l;
                    ml[kTileRows] = l;
                    if (row == 0 && u == 0)
                        p.ws.info[slot] = PartInfo{walk.req, walk.kvh, walk.tok0() * a.group, walk.k1 == walk.total};
                }
            }
            ++piece;
            __syncwarp();
            if (lane == 0) more = place->next();
            more = __shfl_sync(0xffffffffu, more, 0);
            __syncwarp();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, CF::kTmemCols);
    }
    // nothing here needs paged_rows_kernel, which may run beside this one
    wait_for_previous();
}

}  // namespace tiles
}  // namespace paged
}  // namespace ra
