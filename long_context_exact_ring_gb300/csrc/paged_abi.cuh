// paged_abi.cuh -- the C-ABI boundary of the paged key/value cache: argument
// checks and launches.  Part of ring_attn.cu, whose per-device state and
// error reporting it uses.
#pragma once

namespace {

// Strides of `count` dimensions of the given extents, or those of the
// contiguous layout when the caller passes NULL.  Usable are positive
// multiples of 8 elements (16 bytes) below 2^35; the stride of an extent-1
// dimension is never used and becomes 0.
bool paged_strides(long long* out, const long long* given, const long long* contiguous, const int* extents,
                   int count)
{
    for (int x = 0; x < count; ++x) {
        const long long st = given ? given[x] : contiguous[x];
        if (extents[x] <= 1) out[x] = 0;
        else if (st <= 0 || st % 8 != 0 || st >= (1ll << 35)) return false;
        else out[x] = st;
    }
    return true;
}

bool row_strides(long long* out, const long long* given, int tokens, int heads, int d)
{
    const long long contiguous[2] = {(long long)heads * d, d};
    const int extents[2] = {tokens, heads};
    return paged_strides(out, given, contiguous, extents, 2);
}

bool pool_strides(ra::paged::PoolLayout* out, const long long* given, int pages, int page_size, int heads, int d)
{
    const long long contiguous[3] = {(long long)page_size * heads * d, (long long)heads * d, d};
    const int extents[3] = {pages, page_size, heads};
    long long st[3];
    if (!paged_strides(st, given, contiguous, extents, 3)) return false;
    *out = {st[0], st[1], st[2]};
    return true;
}

int check_pool(int num_pages, int page_size, int H_kv, int d)
{
    if (num_pages < 1 || page_size < 1 || H_kv < 1) return RA_ERR_INVALID_ARG;
    if (page_size % 8 != 0 || (d != 64 && d != 128)) return RA_ERR_UNSUPPORTED;
    if ((long long)num_pages * page_size >= (1ll << 31)) return RA_ERR_UNSUPPORTED;
    return RA_OK;
}

// log2 of a power of two, else -1
int page_shift(int page_size)
{
    for (int x = 0; x < 31; ++x)
        if (page_size == (1 << x)) return x;
    return -1;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A kernel that moves registers between its warps waits for ever if it starts
// with fewer than it hands out: refused here, before any launch.
template <typename Kernel>
cudaError_t check_registers(Kernel kernel, int threads, int few, int many)
{
    cudaFuncAttributes attr;
    const cudaError_t e = cudaFuncGetAttributes(&attr, kernel);
    if (e != cudaSuccess) return e;
    return attr.numRegs * threads >= 128 * few + (threads - 128) * many ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <int D, bool kHalf>
cudaError_t configure_attn_kernels()
{
    namespace pr = ra::paged::rows;
    namespace pt = ra::paged::tiles;
    cudaError_t e = check_registers(pr::paged_rows_kernel<D, kHalf>, pr::kThreads, pr::kFewRegs, pr::kManyRegs);
    if (e == cudaSuccess)
        e = check_registers(pt::paged_tiles_kernel<D, kHalf>, pt::kThreads, pt::kFewRegs, pt::kManyRegs);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(pr::paged_rows_kernel<D, kHalf>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 pr::Cfg<D>::kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(pt::paged_tiles_kernel<D, kHalf>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 pt::Cfg<D>::kSmemBytes);
    return e;
}

cudaError_t configure_plan_kernel()
{
    cudaError_t e = cudaFuncSetAttribute(ra::paged::paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)ra::paged::plan_smem(ra::paged::kMaxRequests));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(ra::paged::paged_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
}

cudaError_t configure_all_attn_kernels()
{
    cudaError_t e = configure_attn_kernels<64, false>();
    if (e == cudaSuccess) e = configure_attn_kernels<64, true>();
    if (e == cudaSuccess) e = configure_attn_kernels<128, false>();
    if (e == cudaSuccess) e = configure_attn_kernels<128, true>();
    return e;
}

// Kernels that have to be configured before their first launch on a device.
// No call depends on kernels that it does not launch.
struct Configured {
    cudaError_t (*configure)();
    const char* what;
    std::atomic<bool> ready[kMaxDevices];
};
Configured g_plan_kernel{configure_plan_kernel, "paged_plan_kernel set-up", {}};
Configured g_attn_kernels{configure_all_attn_kernels, "paged attention kernels' set-up", {}};

// device_state, and those kernels configured.
int configured_state(DeviceState** out, Configured& kernels)
{
    const int rc = device_state(out);
    if (rc != RA_OK) return rc;
    std::atomic<bool>& ready = kernels.ready[*out - g_dev];
    if (ready.load(std::memory_order_acquire)) return RA_OK;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!ready.load(std::memory_order_relaxed)) {
        CaptureRelaxed relaxed;      // as in device_state
        const cudaError_t e = kernels.configure();
        if (e != cudaSuccess) return fail_cuda(e, kernels.what);
        ready.store(true, std::memory_order_release);
    }
    return RA_OK;
}

// 4-D tiled map of 2-byte elements with 128-byte swizzle, 64 columns wide.  L2
// fetches whole rows: with d 64, 256 bytes would bring the neighbouring head's
// row too, which another block reads at another time (16 contexts of 8K, 16
// heads: 128 us against 99).  Strides in elements; that of an extent-1 dimension is never stepped along
// and is replaced by a valid one.
int make_paged_map(CUtensorMap* map, const void* ptr, bool half, int d, const int (&extents)[3],
                   const long long (&strides)[3], const int (&box_rows)[3])
{
    cuuint64_t dims[4] = {(cuuint64_t)d, 1, 1, 1}, st[3];
    cuuint32_t box[4] = {64u, 1u, 1u, 1u}, estr[4] = {1u, 1u, 1u, 1u};
    for (int x = 0; x < 3; ++x) {
        dims[x + 1] = (cuuint64_t)extents[x];
        st[x] = (cuuint64_t)(extents[x] > 1 ? strides[x] : d) * 2;
        box[x + 1] = (cuuint32_t)box_rows[x];
    }
    const CUresult r = g_encode(map, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                                const_cast<void*>(ptr), dims, st, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                CU_TENSOR_MAP_SWIZZLE_128B,
                                d == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        std::snprintf(g_last_error, sizeof(g_last_error), "cuTensorMapEncodeTiled (paged) failed (%d)", (int)r);
        return RA_ERR_CUDA;
    }
    return RA_OK;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// A launch that may begin before the kernel in front of it is over
// (`follows`; see let_next_start).
template <typename... Params, typename... Args>
cudaError_t launch_after(bool follows, void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t s,
                         Args... args)
{
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = follows ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Up to 16 packed rows (new tokens x query heads of a key/value head) a
// request is served by paged_rows_kernel, above by paged_tiles_kernel.
constexpr int kFewRows = 16;

// The tensor maps of both kernels; paged_tiles_kernel alone reads Q by one.
struct TileMaps {
    CUtensorMap q, k, v;
};

int make_maps(TileMaps* m, const ra::paged::AttnParams& p, bool half, int d, int tok_tile, int box_rows, bool with_q)
{
    int rc = make_paged_map(&m->k, p.kc, half, d, {p.page_size, p.kv_heads, p.num_pages}, {p.lk.st, p.lk.sh, p.lk.sp},
                            {box_rows, 1, 1});
    if (rc == RA_OK)
        rc = make_paged_map(&m->v, p.vc, half, d, {p.page_size, p.kv_heads, p.num_pages}, {p.lv.st, p.lv.sh, p.lv.sp},
                            {box_rows, 1, 1});
    if (rc == RA_OK && with_q)
        rc = make_paged_map(&m->q, p.q, half, d, {p.group, p.tokens, p.kv_heads},
                            {p.q_head, p.q_tok, p.q_head * p.group}, {p.group, tok_tile, 1});
    return rc;
}

template <int D, bool kHalf>
cudaError_t launch_rows(const TileMaps& maps, const ra::paged::rows::RowsParams& p, int blocks, cudaStream_t s)
{
    namespace pr = ra::paged::rows;
    ra::prof::Scope ps(ra::prof::kPagedRows, s);
    const cudaError_t r = launch_after(false, pr::paged_rows_kernel<D, kHalf>, dim3(blocks), pr::kThreads,
                                       pr::Cfg<D>::kSmemBytes, s, maps.k, maps.v, p);
    ps.done();
    return r;
}

template <int D, bool kHalf>
cudaError_t launch_tiles(bool follows, const TileMaps& maps, const ra::paged::tiles::TileParams& p, int blocks,
                         cudaStream_t s)
{
    namespace pt = ra::paged::tiles;
    ra::prof::Scope ps(ra::prof::kPagedTiles, s);
    const cudaError_t r = launch_after(follows, pt::paged_tiles_kernel<D, kHalf>, dim3(blocks), pt::kThreads,
                                       pt::Cfg<D>::kSmemBytes, s, maps.q, maps.k, maps.v, p);
    ps.done();
    return r;
}

template <int D, bool kHalf>
int launch_attn(const ra::paged::AttnParams& p, void* workspace, int max_q, int blocks, cudaStream_t s)
{
    using namespace ra::paged;
    const Workspace few = ra::paged::workspace(workspace, kRowsTile);
    const Workspace big = ra::paged::workspace(
        static_cast<char*>(workspace) + align256(workspace_bytes(kRowsTile, D)), kBigTile);
    // Both kernels can serve any request, so a wrong hint costs time only: one
    // kernel alone takes them all where no request should have more rows than
    // kFewRows, or all should have max_q tokens.
    bool run_rows = true, run_tiles = true;
    if ((long long)max_q * p.group <= kFewRows || (long long)p.tokens * p.group <= kFewRows) run_tiles = false;
    else if (p.group > kFewRows || (long long)p.n * max_q <= p.tokens) run_rows = false;
    const int box_rows = std::min(p.page_size & -p.page_size, tiles::kBN);
    TileMaps maps;
    const int rc = make_maps(&maps, p, kHalf, D, tiles::kBM / p.group, box_rows, run_tiles);
    if (rc != RA_OK) return rc;
    const rows::RowsParams rp{p, few, {0, run_tiles ? kFewRows : INT_MAX}, box_rows, g_wait_limit_ns.load()};
    const tiles::TileParams tp{p, big, {run_rows ? kFewRows : 0, INT_MAX}, tiles::kBM / p.group, box_rows,
                               g_wait_limit_ns.load()};
    cudaError_t e = cudaSuccess;
    if (run_rows) e = launch_rows<D, kHalf>(maps, rp, blocks, s);
    if (run_tiles && e == cudaSuccess) e = launch_tiles<D, kHalf>(run_rows, maps, tp, blocks, s);
    if (e == cudaSuccess) {
        const int first = run_tiles ? 0 : kBigSlices, last = kBigSlices + (run_rows ? kRowsSlices : 0);
        ra::prof::Scope ps(ra::prof::kPagedJoin, s);
        e = launch_after(true, paged_join_kernel<D, kHalf>, dim3(blocks, last - first), kJoinThreads, 0, s, p, few, big, blocks,
                         tp.tok_tile * p.group, first);
        ps.done();
    }
    if (e != cudaSuccess) cudaGetLastError();    // reported here, not by a later call
    return e == cudaSuccess ? (int)RA_OK : fail_cuda(e, "paged attention launch");
}

}  // namespace

extern "C" {

int paged_kv_plan(const int* seq_lens, const int* new_lens, int n, int* block_table, long long table_stride,
                  int max_pages, int* free_list, int num_pages, const int* counts, int page_size, int tokens,
                  int* seq_lens_out, int* cu_q, int* slots, int* counts_out, void* stream)
{
    if (n < 0 || tokens < 0) return RA_ERR_INVALID_ARG;
    const int rc = check_pool(num_pages, page_size, 1, 64);
    if (rc != RA_OK) return rc;
    if (max_pages < 1 || table_stride < max_pages) return RA_ERR_INVALID_ARG;
    if (n > ra::paged::kMaxRequests || (long long)n * max_pages > (1ll << 30) || num_pages > (1 << 30) ||
        tokens > (1 << 30) || (long long)max_pages * page_size > (1ll << 30))
        return RA_ERR_UNSUPPORTED;
    if (!free_list || !counts || !counts_out || !cu_q || (tokens > 0 && !slots) ||
        (n > 0 && (!seq_lens || !new_lens || !block_table || !seq_lens_out)))
        return RA_ERR_INVALID_ARG;
    const void* all[] = {seq_lens, new_lens, block_table, free_list, counts, seq_lens_out, cu_q, slots, counts_out};
    for (const void* x : all)
        if (!aligned4(x)) return RA_ERR_INVALID_ARG;
    DeviceState* st = nullptr;
    const int e = configured_state(&st, g_plan_kernel);
    if (e != RA_OK) return e;
    ra::paged::PlanParams p{seq_lens,     new_lens, block_table, table_stride, free_list, counts, seq_lens_out,
                            cu_q,         slots,    counts_out,  n,            max_pages, num_pages, page_size,
                            page_shift(page_size), tokens};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t smem = ra::paged::plan_smem(n);
    const unsigned blocks = ra::paged::kPlanCluster;
    cudaError_t ce;
    {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = blocks;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(blocks);
        cfg.blockDim = dim3(ra::paged::kPlanThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        ra::prof::Scope ps(ra::prof::kPagedPlan, s);
        ce = cudaLaunchKernelEx(&cfg, ra::paged::paged_plan_kernel, p);
        ps.done();
    }
    if (ce != cudaSuccess) cudaGetLastError();    // reported here, not by a later call
    return ce == cudaSuccess ? RA_OK : fail_cuda(ce, "paged_plan_kernel launch");
}

int paged_kv_append(const void* k, const long long* k_strides, const void* v, const long long* v_strides,
                    void* k_cache, const long long* k_cache_strides, void* v_cache,
                    const long long* v_cache_strides, const int* slots, int tokens, int H_kv, int d, int num_pages,
                    int page_size, void* stream)
{
    if (tokens < 0) return RA_ERR_INVALID_ARG;
    int rc = check_pool(num_pages, page_size, H_kv, d);
    if (rc != RA_OK) return rc;
    long long ks[2], vs[2];
    ra::paged::PoolLayout lk, lv;
    if (!row_strides(ks, k_strides, tokens, H_kv, d) || !row_strides(vs, v_strides, tokens, H_kv, d) ||
        !pool_strides(&lk, k_cache_strides, num_pages, page_size, H_kv, d) ||
        !pool_strides(&lv, v_cache_strides, num_pages, page_size, H_kv, d))
        return RA_ERR_INVALID_ARG;
    if (tokens == 0) return RA_OK;
    if (!k || !v || !k_cache || !v_cache || !slots) return RA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned4(slots))
        return RA_ERR_INVALID_ARG;
    if (H_kv > (1 << 20)) return RA_ERR_UNSUPPORTED;
    DeviceState* st = nullptr;
    if ((rc = device_state(&st)) != RA_OK) return rc;
    const int vec_shift = d == 128 ? 4 : 3;
    const long long pieces = ((long long)tokens * H_kv) << vec_shift;
    const long long blocks = std::min((pieces + 255) / 256, (long long)st->num_sms * 16);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    ra::prof::Scope ps(ra::prof::kPagedAppend, s);
    ra::paged::paged_append_kernel<<<(unsigned)blocks, 256, 0, s>>>(
        static_cast<const uint16_t*>(k), ks[0], ks[1], static_cast<const uint16_t*>(v), vs[0], vs[1],
        static_cast<uint16_t*>(k_cache), lk, static_cast<uint16_t*>(v_cache), lv, slots, tokens, H_kv, vec_shift,
        page_size, num_pages * page_size, st->status);
    ps.done();
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? RA_OK : fail_cuda(e, "paged_append_kernel launch");
}

size_t paged_attn_workspace_size(int n, int tokens, int H, int H_kv, int d)
{
    if (n <= 0 || tokens <= 0 || H <= 0 || H_kv <= 0 || H % H_kv != 0 || (d != 64 && d != 128)) return 0;
    const size_t few = align256(ra::paged::workspace_bytes(ra::paged::rows::kRows, d));
    if ((long long)tokens * (H / H_kv) <= kFewRows) return few;
    return few + align256(ra::paged::workspace_bytes(ra::paged::tiles::kTileRows, d));
}

int paged_attn_fwd(const void* q, const long long* q_strides, const void* k_cache, const long long* k_cache_strides,
                   const void* v_cache, const long long* v_cache_strides, const int* block_table,
                   long long table_stride, const int* seq_lens, const int* cu_q, void* o, const long long* o_strides,
                   float* lse, int dtype, int n, int tokens, int H, int H_kv, int d, int num_pages, int page_size,
                   int max_pages, int max_q, int causal, float scale, void* workspace, size_t workspace_bytes,
                   void* stream)
{
    if (n < 0 || tokens < 0 || H < 1 || max_q < 0 || (causal != 0 && causal != 1)) return RA_ERR_INVALID_ARG;
    if (dtype != RA_BF16 && dtype != RA_FP16) return RA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.f)) return RA_ERR_INVALID_ARG;
    int rc = check_pool(num_pages, page_size, H_kv, d);
    if (rc != RA_OK) return rc;
    if (H % H_kv != 0 || max_pages < 1 || table_stride < max_pages) return RA_ERR_INVALID_ARG;
    if (H / H_kv > 128 || H > (1 << 20) || (long long)H * tokens >= (1ll << 31) ||
        (long long)max_pages * page_size > (1ll << 30))
        return RA_ERR_UNSUPPORTED;
    long long qs[2], os[2];
    ra::paged::PoolLayout lk, lv;
    if (!row_strides(qs, q_strides, tokens, H, d) || !row_strides(os, o_strides, tokens, H, d) ||
        !pool_strides(&lk, k_cache_strides, num_pages, page_size, H_kv, d) ||
        !pool_strides(&lv, v_cache_strides, num_pages, page_size, H_kv, d))
        return RA_ERR_INVALID_ARG;
    if (n == 0 || tokens == 0) return RA_OK;
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !cu_q || !o || !lse || !workspace)
        return RA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned4(block_table) ||
        !aligned4(seq_lens) || !aligned4(cu_q) || !aligned4(lse) || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < paged_attn_workspace_size(n, tokens, H, H_kv, d))
        return RA_ERR_INVALID_ARG;
    DeviceState* st = nullptr;
    if ((rc = configured_state(&st, g_attn_kernels)) != RA_OK) return rc;

    ra::paged::AttnParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.q_tok = qs[0];
    p.q_head = qs[1];
    p.kc = static_cast<const uint16_t*>(k_cache);
    p.lk = lk;
    p.vc = static_cast<const uint16_t*>(v_cache);
    p.lv = lv;
    p.table = block_table;
    p.table_stride = table_stride;
    p.seq_lens = seq_lens;
    p.cu_q = cu_q;
    p.o = static_cast<uint16_t*>(o);
    p.o_tok = os[0];
    p.o_head = os[1];
    p.lse = lse;
    p.n = n;
    p.tokens = tokens;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.page_shift = page_shift(page_size);
    p.kv_heads = H_kv;
    p.group = H / H_kv;
    p.causal = causal;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    p.status = st->status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int blocks = std::min(st->num_sms, ra::paged::kMaxBlocks);
    if (d == 128)
        return dtype == RA_FP16 ? launch_attn<128, true>(p, workspace, max_q, blocks, s)
                                : launch_attn<128, false>(p, workspace, max_q, blocks, s);
    return dtype == RA_FP16 ? launch_attn<64, true>(p, workspace, max_q, blocks, s)
                            : launch_attn<64, false>(p, workspace, max_q, blocks, s);
}

}  // extern "C"
