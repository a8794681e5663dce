// rope_abi.cuh -- the C-ABI boundary of the norm and rotation of queries and
// keys: argument checks and launches.  Part of ring_attn.cu, behind
// paged_abi.cuh, whose helpers it uses.
#pragma once

namespace {

int check_rope(int dtype, int heads_a, int heads_b, int d, int rot, int interleaved, float eps, float amplitude)
{
    if (dtype != RA_BF16 && dtype != RA_FP16) return RA_ERR_INVALID_ARG;
    if (heads_a < 0 || heads_b < 0 || (interleaved != 0 && interleaved != 1)) return RA_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(amplitude)) return RA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return RA_ERR_UNSUPPORTED;
    if (rot < 2 || rot > d || rot % 2 != 0) return RA_ERR_INVALID_ARG;
    if (rot % 16 != 0 || heads_a > (1 << 20) || heads_b > (1 << 20)) return RA_ERR_UNSUPPORTED;
    return RA_OK;
}

// Shares of a token's `rows` rows: one where the tokens alone occupy the warps of
// the forward kernel, else as many as that takes, of at least one row to a lane
// group (a decode token, 32 heads over 8: 4.0 us, with whole batches 4.7).  The
// backward kernel takes the same shares with three quarters of the warps.
int rope_parts(int tokens, int rows, int d, int sms)
{
    const int step = 512 / d;
    const long long want = ((long long)sms * ra::rope::kWarps * ra::rope::kBlocksPerSm + tokens - 1) / tokens;
    return (int)std::max(1ll, std::min(want, (long long)(rows + step - 1) / step));
}

int rope_blocks(int tokens, int parts, int sms, int per_sm)
{
    const long long blocks = ((long long)tokens * parts + ra::rope::kWarps - 1) / ra::rope::kWarps;
    return (int)std::min(blocks, (long long)std::min(sms, 160) * per_sm);
}

template <int D, bool kHalf, bool kPaged>
void launch_rope_fwd(const ra::rope::Params& p, const ra::rope::Paged& c, int blocks, cudaStream_t s)
{
    using namespace ra::rope;
    if (p.interleaved) rope_fwd_kernel<D, kHalf, true, kPaged><<<blocks, kThreads, 0, s>>>(p, c);
    else rope_fwd_kernel<D, kHalf, false, kPaged><<<blocks, kThreads, 0, s>>>(p, c);
}

template <bool kPaged>
int launch_rope_fwd(const ra::rope::Params& p, const ra::rope::Paged& c, int d, bool half, int blocks, cudaStream_t s)
{
    ra::prof::Scope ps(ra::prof::kRopeFwd, s);
    if (d == 128 && half) launch_rope_fwd<128, true, kPaged>(p, c, blocks, s);
    else if (d == 128) launch_rope_fwd<128, false, kPaged>(p, c, blocks, s);
    else if (half) launch_rope_fwd<64, true, kPaged>(p, c, blocks, s);
    else launch_rope_fwd<64, false, kPaged>(p, c, blocks, s);
    ps.done();
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? RA_OK : fail_cuda(e, "rope_fwd_kernel launch");
}

template <int D, bool kHalf>
void launch_rope_bwd(const ra::rope::Params& p, int blocks, cudaStream_t s)
{
    using namespace ra::rope;
    if (p.interleaved) rope_bwd_kernel<D, kHalf, true><<<blocks, kThreads, 0, s>>>(p);
    else rope_bwd_kernel<D, kHalf, false><<<blocks, kThreads, 0, s>>>(p);
}

// A tensor's rows from the caller's strides (batch, head, position); false if
// they cannot be used.
bool rope_rows(const void* ptr, const long long* strides, int B, int heads, int S, int d, const uint16_t** out,
               long long* b, long long* s, long long* h)
{
    ra::RowLayout l = layout_from(strides, heads, S, d);
    if (heads == 0) l = ra::RowLayout{0, 0, 0};      // no rows: nothing is read
    else if (!layout_ok(l, B, heads, S)) return false;
    *out = static_cast<const uint16_t*>(ptr);
    *b = l.sb;
    *s = l.ss;
    *h = l.sh;
    return true;
}

}  // namespace

extern "C" {

int qk_norm_rope_fwd(const void* q, const long long* q_strides, const void* k, const long long* k_strides,
                     const float* q_weight, const float* k_weight, float eps, const int* positions, int per_batch,
                     const float* inv_freq, int rot_dim, int interleaved, float amplitude, void* q_out,
                     const long long* q_out_strides, void* k_out, const long long* k_out_strides, int dtype, int B,
                     int H, int H_kv, int S, int d, void* stream)
{
    int rc = check_rope(dtype, H, H_kv, d, rot_dim, interleaved, eps, amplitude);
    if (rc != RA_OK) return rc;
    if (B < 0 || S < 0 || (per_batch != 0 && per_batch != 1)) return RA_ERR_INVALID_ARG;
    if ((long long)B * S >= (1ll << 31)) return RA_ERR_UNSUPPORTED;
    if (B == 0 || S == 0 || H + H_kv == 0) return RA_OK;
    ra::rope::Params p = {};
    const uint16_t* out;
    if (!rope_rows(q, q_strides, B, H, S, d, &p.q.x, &p.q.xb, &p.q.xs, &p.q.xh) ||
        !rope_rows(k, k_strides, B, H_kv, S, d, &p.k.x, &p.k.xb, &p.k.xs, &p.k.xh))
        return RA_ERR_INVALID_ARG;
    if (!rope_rows(q_out, q_out_strides, B, H, S, d, &out, &p.q.ob, &p.q.os, &p.q.oh)) return RA_ERR_INVALID_ARG;
    p.q.out = const_cast<uint16_t*>(out);
    if (!rope_rows(k_out, k_out_strides, B, H_kv, S, d, &out, &p.k.ob, &p.k.os, &p.k.oh)) return RA_ERR_INVALID_ARG;
    p.k.out = const_cast<uint16_t*>(out);
    if (!positions || !inv_freq || (H > 0 && (!q || !q_out)) || (H_kv > 0 && (!k || !k_out))) return RA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned4(positions) ||
        !aligned4(inv_freq) || !aligned4(q_weight) || !aligned4(k_weight))
        return RA_ERR_INVALID_ARG;
    DeviceState* st = nullptr;
    if ((rc = device_state(&st)) != RA_OK) return rc;
    p.q.w = q_weight;
    p.k.w = k_weight;
    p.q.heads = H;
    p.k.heads = H_kv;
    p.positions = positions;
    p.pos_batch = per_batch ? S : 0;
    p.inv_freq = inv_freq;
    p.eps = eps;
    p.amplitude = amplitude;
    p.sign = 1.f;
    p.rot = rot_dim;
    p.interleaved = interleaved;
    p.S = S;
    p.tokens = B * S;
    p.parts = rope_parts(p.tokens, H + H_kv, d, st->num_sms);
    return launch_rope_fwd<false>(p, ra::rope::Paged{}, d, dtype == RA_FP16,
                                  rope_blocks(p.tokens, p.parts, st->num_sms, ra::rope::kBlocksPerSm),
                                  static_cast<cudaStream_t>(stream));
}

size_t qk_norm_rope_bwd_workspace_size(int d)
{
    if (d != 64 && d != 128) return 0;
    return (size_t)ra::rope::kMaxBlocks * 2 * d * sizeof(float);
}

int qk_norm_rope_bwd(const void* dq, const long long* dq_strides, const void* dk, const long long* dk_strides,
                     const void* q, const long long* q_strides, const void* k, const long long* k_strides,
                     const float* q_weight, const float* k_weight, float eps, const int* positions, int per_batch,
                     const float* inv_freq, int rot_dim, int interleaved, float amplitude, void* dq_in,
                     const long long* dq_in_strides, void* dk_in, const long long* dk_in_strides, float* dq_weight,
                     float* dk_weight, int dtype, int B, int H, int H_kv, int S, int d, void* workspace,
                     size_t workspace_bytes, void* stream)
{
    using namespace ra::rope;
    int rc = check_rope(dtype, H, H_kv, d, rot_dim, interleaved, eps, amplitude);
    if (rc != RA_OK) return rc;
    if (B < 0 || S < 0 || (per_batch != 0 && per_batch != 1)) return RA_ERR_INVALID_ARG;
    if ((long long)B * S >= (1ll << 31)) return RA_ERR_UNSUPPORTED;
    // a weight and its gradient come together
    if (!q_weight != !dq_weight || !k_weight != !dk_weight) return RA_ERR_INVALID_ARG;
    const bool norm = q_weight || k_weight, rows = B > 0 && S > 0 && H + H_kv > 0;
    if (!rows && !norm) return RA_OK;
    Params p = {};
    if (!aligned4(q_weight) || !aligned4(k_weight) || !aligned4(dq_weight) || !aligned4(dk_weight))
        return RA_ERR_INVALID_ARG;
    if (rows) {
        const uint16_t* out;
        if (!rope_rows(dq, dq_strides, B, H, S, d, &p.q.g, &p.q.gb, &p.q.gs, &p.q.gh) ||
            !rope_rows(dk, dk_strides, B, H_kv, S, d, &p.k.g, &p.k.gb, &p.k.gs, &p.k.gh))
            return RA_ERR_INVALID_ARG;
        // without a norm the gradient does not depend on the rows
        if ((q_weight && !rope_rows(q, q_strides, B, H, S, d, &p.q.x, &p.q.xb, &p.q.xs, &p.q.xh)) ||
            (k_weight && !rope_rows(k, k_strides, B, H_kv, S, d, &p.k.x, &p.k.xb, &p.k.xs, &p.k.xh)))
            return RA_ERR_INVALID_ARG;
        if (!rope_rows(dq_in, dq_in_strides, B, H, S, d, &out, &p.q.ob, &p.q.os, &p.q.oh)) return RA_ERR_INVALID_ARG;
        p.q.out = const_cast<uint16_t*>(out);
        if (!rope_rows(dk_in, dk_in_strides, B, H_kv, S, d, &out, &p.k.ob, &p.k.os, &p.k.oh)) return RA_ERR_INVALID_ARG;
        p.k.out = const_cast<uint16_t*>(out);
        if (!positions || !inv_freq || (H > 0 && (!dq || !dq_in || (q_weight && !q))) ||
            (H_kv > 0 && (!dk || !dk_in || (k_weight && !k))))
            return RA_ERR_INVALID_ARG;
        if (!aligned16(dq) || !aligned16(dk) || !aligned16(dq_in) || !aligned16(dk_in) || !aligned4(positions) ||
            !aligned4(inv_freq) || (q_weight && !aligned16(q)) || (k_weight && !aligned16(k)))
            return RA_ERR_INVALID_ARG;
        if (norm && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
                     workspace_bytes < qk_norm_rope_bwd_workspace_size(d)))
            return RA_ERR_INVALID_ARG;
    }
    DeviceState* st = nullptr;
    if ((rc = device_state(&st)) != RA_OK) return rc;
    p.q.w = q_weight;
    p.k.w = k_weight;
    p.q.heads = H;
    p.k.heads = H_kv;
    p.positions = positions;
    p.pos_batch = per_batch ? S : 0;
    p.inv_freq = inv_freq;
    p.eps = eps;
    p.amplitude = amplitude;
    p.sign = -1.f;
    p.rot = rot_dim;
    p.interleaved = interleaved;
    p.S = S;
    p.tokens = B * S;
    p.partial = norm ? static_cast<float*>(workspace) : nullptr;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!norm) {      // a rotation back and nothing else
        p.q.x = p.q.g;
        p.q.xb = p.q.gb;
        p.q.xs = p.q.gs;
        p.q.xh = p.q.gh;
        p.k.x = p.k.g;
        p.k.xb = p.k.gb;
        p.k.xs = p.k.gs;
        p.k.xh = p.k.gh;
        p.parts = rope_parts(p.tokens, H + H_kv, d, st->num_sms);
        return launch_rope_fwd<false>(p, Paged{}, d, dtype == RA_FP16,
                                      rope_blocks(p.tokens, p.parts, st->num_sms, kBlocksPerSm), s);
    }
    int blocks = 0;
    cudaError_t e = cudaSuccess;
    if (rows) {
        p.parts = rope_parts(p.tokens, H + H_kv, d, st->num_sms);
        blocks = rope_blocks(p.tokens, p.parts, st->num_sms, kBackPerSm);
        ra::prof::Scope ps(ra::prof::kRopeBwd, s);
        const bool half = dtype == RA_FP16;
        if (d == 128 && half) launch_rope_bwd<128, true>(p, blocks, s);
        else if (d == 128) launch_rope_bwd<128, false>(p, blocks, s);
        else if (half) launch_rope_bwd<64, true>(p, blocks, s);
        else launch_rope_bwd<64, false>(p, blocks, s);
        ps.done();
        e = cudaGetLastError();
    }
    if (norm && e == cudaSuccess) {
        ra::prof::Scope ps(ra::prof::kRopeWeights, s);
        e = launch_after(rows, rope_weight_grad_kernel, dim3(d / kWarps, 2), kThreads, 0, s,
                         (const float*)p.partial, blocks, d, dq_weight, dk_weight);
        ps.done();
        if (e != cudaSuccess) cudaGetLastError();    // reported here, not by a later call
    }
    return e == cudaSuccess ? RA_OK : fail_cuda(e, "qk_norm_rope_bwd launch");
}

int paged_kv_append_rope(const void* q, const long long* q_strides, const void* k, const long long* k_strides,
                         const void* v, const long long* v_strides, const float* q_weight, const float* k_weight,
                         float eps, const float* inv_freq, int rot_dim, int interleaved, float amplitude, void* q_out,
                         const long long* q_out_strides, void* k_cache, const long long* k_cache_strides,
                         void* v_cache, const long long* v_cache_strides, const int* slots, const int* seq_lens,
                         const int* cu_q, int dtype, int n, int tokens, int H, int H_kv, int d, int num_pages,
                         int page_size, void* stream)
{
    if (n < 0 || tokens < 0 || H < 1) return RA_ERR_INVALID_ARG;
    int rc = check_rope(dtype, H, H_kv, d, rot_dim, interleaved, eps, amplitude);
    if (rc == RA_OK) rc = check_pool(num_pages, page_size, H_kv, d);
    if (rc != RA_OK) return rc;
    long long qs[2], ks[2], vs[2], os[2];
    ra::rope::Paged c = {};
    if (!row_strides(qs, q_strides, tokens, H, d) || !row_strides(ks, k_strides, tokens, H_kv, d) ||
        !row_strides(vs, v_strides, tokens, H_kv, d) || !row_strides(os, q_out_strides, tokens, H, d) ||
        !pool_strides(&c.lk, k_cache_strides, num_pages, page_size, H_kv, d) ||
        !pool_strides(&c.lv, v_cache_strides, num_pages, page_size, H_kv, d))
        return RA_ERR_INVALID_ARG;
    if (n == 0 || tokens == 0) return RA_OK;
    if (!q || !k || !v || !q_out || !k_cache || !v_cache || !inv_freq || !slots || !seq_lens || !cu_q)
        return RA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_cache) ||
        !aligned16(v_cache) || !aligned4(inv_freq) || !aligned4(q_weight) || !aligned4(k_weight) ||
        !aligned4(slots) || !aligned4(seq_lens) || !aligned4(cu_q))
        return RA_ERR_INVALID_ARG;
    DeviceState* st = nullptr;
    if ((rc = device_state(&st)) != RA_OK) return rc;
    ra::rope::Params p = {};
    p.q.x = static_cast<const uint16_t*>(q);
    p.q.xs = qs[0];
    p.q.xh = qs[1];
    p.q.out = static_cast<uint16_t*>(q_out);
    p.q.os = os[0];
    p.q.oh = os[1];
    p.q.w = q_weight;
    p.q.heads = H;
    p.k.x = static_cast<const uint16_t*>(k);
    p.k.xs = ks[0];
    p.k.xh = ks[1];
    p.k.w = k_weight;
    p.k.heads = H_kv;
    p.inv_freq = inv_freq;
    p.eps = eps;
    p.amplitude = amplitude;
    p.sign = 1.f;
    p.rot = rot_dim;
    p.interleaved = interleaved;
    p.S = p.tokens = tokens;
    p.parts = rope_parts(tokens, H + 2 * H_kv, d, st->num_sms);
    c.v = static_cast<const uint16_t*>(v);
    c.vs = vs[0];
    c.vh = vs[1];
    c.kc = static_cast<uint16_t*>(k_cache);
    c.vc = static_cast<uint16_t*>(v_cache);
    c.slots = slots;
    c.seq_lens = seq_lens;
    c.cu_q = cu_q;
    c.n = n;
    c.page_size = page_size;
    c.num_slots = num_pages * page_size;
    c.status = st->status;
    return launch_rope_fwd<true>(p, c, d, dtype == RA_FP16, rope_blocks(tokens, p.parts, st->num_sms, ra::rope::kBlocksPerSm),
                                 static_cast<cudaStream_t>(stream));
}

}  // extern "C"
