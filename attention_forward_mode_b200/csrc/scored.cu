// scored.cu -- host side of the score-modified attention + JVP (tanh cap,
// distance bias, an interval of visible keys per query row, shared key heads):
// attn_jvp_fwd_scored, attn_jvp_fwd_scored_stats, attn_jvp_bwd_scored.
// Argument checks, tensor maps, launches; no device memory is allocated here.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "attn_jvp.h"
#include "host_common.h"
#include "jvp_bwd_sm100.cuh"
#include "jvp_sm100.cuh"
#include "selftest_sm100.cuh"

using namespace ajvp;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
// positions are exact in fp32, which the distance bias computes in
constexpr int64_t kMaxLen = int64_t(1) << 24;

struct Setup {
    std::once_flag once;
    cudaError_t error = cudaSuccess;
};
Setup g_setup[host::kMaxDevices];

template <int MASK>
cudaError_t set_fwd() {
    return cudaFuncSetAttribute(sm100::attn_jvp_fwd_kernel<false, MASK, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sm100::SMEM_BYTES);
}
template <int MASK, bool kSplitK>
cudaError_t set_bwd() {
    return cudaFuncSetAttribute(bwd::attn_jvp_bwd_scored_kernel<MASK, kSplitK>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bwd::SMEM_ALL);
}
template <int MASK>
cudaError_t set_mask() {
    cudaError_t e = set_fwd<MASK>();
    if (e == cudaSuccess) e = set_bwd<MASK, false>();
    if (e == cudaSuccess) e = set_bwd<MASK, true>();
    return e;
}

int setup(int *dev) {
    int rc = host::device(dev);
    if (rc != AJVP_OK) return rc;
    Setup &s = g_setup[*dev];
    std::call_once(s.once, [&]() {
        s.error = set_mask<MASK_SCORED>();
        if (s.error == cudaSuccess) s.error = set_mask<MASK_SCORED | MASK_CAP>();
        if (s.error == cudaSuccess) s.error = set_mask<MASK_SCORED | MASK_BIAS>();
        if (s.error == cudaSuccess) s.error = set_mask<MASK_SCORED | MASK_CAP | MASK_BIAS>();
        if (s.error == cudaSuccess) s.error = set_fwd<MASK_SCORED | MASK_CAP | MASK_FIXED>();
        if (s.error == cudaSuccess) s.error = set_fwd<MASK_SCORED | MASK_CAP | MASK_BIAS | MASK_FIXED>();
    });
    return s.error == cudaSuccess ? AJVP_OK : host::fail(s.error);
}

struct Sizes {
    int64_t B, H, Hkv, Lq, Lk, d;
};

int check_sizes(const Sizes &z, float scale, float softcap) {
    if (z.B < 0 || z.H < 0 || z.Hkv < 0 || z.Lq < 0 || z.Lk < 1 || z.d < 1) return AJVP_ERR_INVALID_ARG;
    if (z.H > 0 && (z.Hkv < 1 || z.H % z.Hkv != 0)) return AJVP_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f) return AJVP_ERR_INVALID_ARG;
    if (softcap > 0.f && (!std::isfinite(2.f * scale * kLog2e / softcap) || !std::isfinite(2.f / softcap) ||
                          !std::isfinite(softcap * kLog2e)))
        return AJVP_ERR_INVALID_ARG;
    return AJVP_OK;
}

int check_large(const Sizes &z) {
    if (z.Lq >= kMaxLen || z.Lk >= kMaxLen || z.B >= (int64_t(1) << 31) || z.H >= (int64_t(1) << 31) ||
        z.B * z.H >= (int64_t(1) << 31))
        return AJVP_ERR_TOO_LARGE;
    if ((z.Lq + 127) / 128 * z.B * z.H >= (int64_t(1) << 31) || (z.Lk + 127) / 128 * z.B * z.H >= (int64_t(1) << 31))
        return AJVP_ERR_TOO_LARGE;
    return AJVP_OK;
}

Score make_score(const Sizes &z, float scale, float softcap, const float *slopes, const int32_t *begin,
                 const int32_t *end) {
    Score s;
    std::memset(&s, 0, sizeof(s));
    s.begin = begin;
    s.end = end;
    s.slopes = slopes;
    if (softcap > 0.f) {
        s.cap_in = 2.f * scale * kLog2e / softcap;
        s.cap_w = scale / softcap;
        s.cap_out = softcap * kLog2e;
        s.cap_second = 2.f / softcap;
    }
    s.H = (int)z.H;
    s.Hkv = (int)z.Hkv;
    s.group = (int)(z.H / z.Hkv);
    return s;
}

int mask_bits(float softcap, const float *slopes) {
    return MASK_SCORED | (softcap > 0.f ? MASK_CAP : 0) | (slopes ? MASK_BIAS : 0);
}

// f(std::integral_constant<int, MASK>) for the run-time mask
template <class F>
int with_mask(int mask, F f) {
    switch (mask) {
        case MASK_SCORED: return f(std::integral_constant<int, MASK_SCORED>());
        case MASK_SCORED | MASK_CAP: return f(std::integral_constant<int, MASK_SCORED | MASK_CAP>());
        case MASK_SCORED | MASK_BIAS: return f(std::integral_constant<int, MASK_SCORED | MASK_BIAS>());
        default: return f(std::integral_constant<int, MASK_SCORED | MASK_CAP | MASK_BIAS>());
    }
}

// (batch, head) slabs scheduled together: their streamed tensors, four of
// `rows` rows each, take about 100 of the 126 MB of L2 (smaller groups end in a longer
// tail: 12 heads of 8190 under a causal mask, four at a time, 500 instead of 458 us)
int slabs_together(int64_t rows, int64_t BH) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(BH, (100 << 20) / (rows * bwd::HD * 8 + 1)));
}

int fwd_scored(const void *q, const void *k, const void *v, const void *tq, const void *tk, const void *tv, void *o,
               void *to, float *lse, float *mu, const float *slopes, const int32_t *key_begin, const int32_t *key_end,
               const Sizes &z, float scale, float softcap, void *stream) {
    int rc = check_sizes(z, scale, softcap);
    if (rc != AJVP_OK) return rc;
    if (z.B == 0 || z.H == 0 || z.Lq == 0) return AJVP_OK;
    if (!q || !k || !v || !tq || !tk || !tv || !o || !to) return AJVP_ERR_INVALID_ARG;
    if ((rc = check_large(z)) != AJVP_OK) return rc;
    if (z.d != sm100::HD) return AJVP_ERR_UNSUPPORTED_DIM;
    for (const void *p : {q, k, v, tq, tk, tv, (const void *)o, (const void *)to, (const void *)lse, (const void *)mu})
        if (!host::aligned(p, 16)) return AJVP_ERR_MISALIGNED;
    for (const void *p : {(const void *)slopes, (const void *)key_begin, (const void *)key_end})
        if (!host::aligned(p, 4)) return AJVP_ERR_MISALIGNED;
    int dev = 0;
    if ((rc = setup(&dev)) != AJVP_OK) return rc;
    if ((rc = host::encoder()) != AJVP_OK) return rc;

    const int64_t BH = z.B * z.H, BHk = z.B * z.Hkv;
    sm100::Params p;
    std::memset(&p, 0, sizeof(p));
    if ((rc = host::encode(&p.tm_q, q, z.d, z.Lq, BH, 128)) != AJVP_OK) return rc;
    if ((rc = host::encode(&p.tm_tq, tq, z.d, z.Lq, BH, 128)) != AJVP_OK) return rc;
    if ((rc = host::encode(&p.tm_k, k, z.d, z.Lk, BHk, 64)) != AJVP_OK) return rc;
    if ((rc = host::encode(&p.tm_tk, tk, z.d, z.Lk, BHk, 64)) != AJVP_OK) return rc;
    if ((rc = host::encode(&p.tm_v, v, z.d, z.Lk, BHk, 64)) != AJVP_OK) return rc;
    if ((rc = host::encode(&p.tm_tv, tv, z.d, z.Lk, BHk, 64)) != AJVP_OK) return rc;
    if ((rc = host::encode(&p.tm_o, o, z.d, z.Lq, BH, 128)) != AJVP_OK) return rc;
    if ((rc = host::encode(&p.tm_to, to, z.d, z.Lq, BH, 128)) != AJVP_OK) return rc;
    p.lse = lse;
    p.mu = mu;
    p.o_bf = static_cast<__nv_bfloat16 *>(o);
    p.to_bf = static_cast<__nv_bfloat16 *>(to);
    p.BH = (int)BH;
    p.Lq = (int)z.Lq;
    p.Lk = (int)z.Lk;
    p.n_qtiles = (int)((z.Lq + sm100::BR - 1) / sm100::BR);
    p.scale = scale;
    // hidden keys hold +-infinity in units of 1 / scale_log2, which must not be zero
    p.scale_log2 = scale == 0.f ? 1e-30f : scale * kLog2e;
    p.bound_ns = host::wait_bound_ns();
    p.score = make_score(z, scale, softcap, slopes, key_begin, key_end);
    // heads of a group share their keys (and never more slabs than there are: the kernel multiplies them by its row tiles)
    p.score.slabs = (int)std::min<int64_t>(BH, z.H / z.Hkv * slabs_together(z.Lk, BHk));
    return with_mask(mask_bits(softcap, slopes), [&](auto mask) {
        constexpr int M = decltype(mask)::value;
        const dim3 grid((unsigned)(p.n_qtiles * BH));
        if ((M & MASK_CAP) != 0 && p.score.cap_out <= FIXED_CAP)
            sm100::attn_jvp_fwd_kernel<false, (M & MASK_CAP) != 0 ? M | MASK_FIXED : M, true>
                <<<grid, sm100::NTHREADS, sm100::SMEM_BYTES, (cudaStream_t)stream>>>(p);
        else
            sm100::attn_jvp_fwd_kernel<false, M, true>
                <<<grid, sm100::NTHREADS, sm100::SMEM_BYTES, (cudaStream_t)stream>>>(p);
        const cudaError_t e = cudaGetLastError();
        return e == cudaSuccess ? AJVP_OK : host::fail(e);
    });
}

uint64_t range_bytes(int64_t B, int64_t Lk) {
    return ((uint64_t)B * (uint64_t)((Lk + 127) / 128) * sizeof(int2) + 255u) / 256u * 256u;
}

// Parts of a key-side CTA's streamed queries (the 64-row tiles of every head of
// its group).  All three variants share one launch of one CTA per SM, heaviest
// CTAs first, so the run takes about the whole work over the SMs and half of
// the longest CTA: tiles streamed, each with a fixed cost of about eight tiles
// per CTA, plus the partial sums' traffic (2 KB per key and part, a tile's time
// moving some 14 MB).  Splits when that is shorter; ties go to fewer parts.
int64_t split_parts(const Sizes &z, int sm_count) {
    const double fixed = 8.0, mb14 = 14e6;
    const double q_tiles = (double)((z.Lk + bwd::BN - 1) / bwd::BN);
    const double q_ctas = (double)((z.Lq + bwd::BM - 1) / bwd::BM * z.B * z.H);
    const int64_t k_tiles = (z.Lq + bwd::BN - 1) / bwd::BN * (z.H / z.Hkv);
    const double k_ctas = (double)((z.Lk + bwd::BM - 1) / bwd::BM * z.B * z.Hkv);
    int64_t best = 1;
    double best_t = 0.0;
    for (int64_t s = 1; s <= 16 && s <= k_tiles; ++s) {
        const double chunk = (double)((k_tiles + s - 1) / s);
        const double work = q_ctas * (q_tiles + fixed) + 2.0 * k_ctas * (double)s * (chunk + fixed);
        const double longest = std::max(q_tiles, chunk) + fixed;
        const double sums = s > 1 ? (double)s * (double)(z.B * z.Hkv * z.Lk) * 4096.0 / mb14 : 0.0;
        const double t = work / (double)sm_count + 0.5 * longest + sums;
        if (s == 1 || t < best_t * 0.999) {
            best = s;
            best_t = t;
        }
    }
    return best;
}

// Parameters of one backward variant: r resident, l the long and s the short
// streamed pair, out scaled by sc; n_split > 1: partial sums to `partial`
int bwd_params(bwd::Params *p, std::initializer_list<const void *> r, std::initializer_list<const void *> l,
               std::initializer_list<const void *> s, void *out0, void *out1, float sc, const Score &score,
               const void *stats, int64_t BHrow, int64_t BHcol, int64_t Lrow, int64_t Lcol, int64_t Lq, float scale,
               int64_t n_split, float *partial) {
    using namespace ajvp::bwd;
    std::memset(p, 0, sizeof(*p));
    int rc, i = 0;
    for (const void *x : r)
        if ((rc = host::encode(&p->tm_r[i++], x, HD, Lrow, BHrow, 128)) != AJVP_OK) return rc;
    i = 0;
    for (const void *x : l)
        if ((rc = host::encode(&p->tm_l[i++], x, HD, Lcol, BHcol, 64)) != AJVP_OK) return rc;
    i = 0;
    for (const void *x : s)
        if ((rc = host::encode(&p->tm_s[i++], x, HD, Lcol, BHcol, 64)) != AJVP_OK) return rc;
    if ((rc = host::encode(&p->tm_out[0], out0, HD, Lrow, BHrow, 128)) != AJVP_OK) return rc;
    if ((rc = host::encode(&p->tm_out[1], out1, HD, Lrow, BHrow, 128)) != AJVP_OK) return rc;
    p->out_scale[0] = p->out_scale[1] = sc;
    p->BH = (int)BHrow;
    p->n_split = (int)n_split;
    p->partial = partial;
    p->stats = static_cast<const float4 *>(stats);
    p->Lrow = (int)Lrow;
    p->Lcol = (int)Lcol;
    p->Lq = (int)Lq;
    p->n_rtiles = (int)((Lrow + BM - 1) / BM);
    p->scale = scale;
    p->scale_log2 = scale * kLog2e;
    p->bound_ns = host::wait_bound_ns();
    p->score = score;
    p->score.slabs = slabs_together(Lcol * (BHcol > BHrow ? BHcol / BHrow : 1), BHrow);
    return AJVP_OK;
}

}  // namespace

namespace ajvp {
namespace host {
cudaError_t scored_selftest(uint64_t bound_ns, cudaStream_t stream) { return selftest_wait(bound_ns, true, stream); }
cudaError_t scored_status(int *word) {
    int w = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&w, g_status_word, sizeof(int));
    if (e != cudaSuccess || w == 0) return e;
    *word |= w;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_status_word, &zero, sizeof(int));
}
}  // namespace host
}  // namespace ajvp

extern "C" {

int attn_jvp_fwd_scored(const void *q, const void *k, const void *v, const void *tq, const void *tk, const void *tv,
                        void *o, void *to, float *lse, const float *slopes, const int32_t *key_begin,
                        const int32_t *key_end, int64_t B, int64_t H, int64_t Hkv, int64_t Lq, int64_t Lk, int64_t d,
                        float scale, float softcap, void *stream) {
    return fwd_scored(q, k, v, tq, tk, tv, o, to, lse, nullptr, slopes, key_begin, key_end, {B, H, Hkv, Lq, Lk, d},
                      scale, softcap, stream);
}

int attn_jvp_fwd_scored_stats(const void *q, const void *k, const void *v, const void *tq, const void *tk,
                              const void *tv, void *o, void *to, float *lse, float *mu, const float *slopes,
                              const int32_t *key_begin, const int32_t *key_end, int64_t B, int64_t H, int64_t Hkv,
                              int64_t Lq, int64_t Lk, int64_t d, float scale, float softcap, void *stream) {
    if (B > 0 && H > 0 && Lq > 0 && (!lse || !mu)) return AJVP_ERR_INVALID_ARG;
    return fwd_scored(q, k, v, tq, tk, tv, o, to, lse, mu, slopes, key_begin, key_end, {B, H, Hkv, Lq, Lk, d}, scale,
                      softcap, stream);
}

uint64_t attn_jvp_bwd_scored_workspace_bytes(int64_t B, int64_t H, int64_t Hkv, int64_t Lq, int64_t Lk) {
    const Sizes z{B, H, Hkv, Lq, Lk, bwd::HD};
    if (check_sizes(z, 1.f, 0.f) != AJVP_OK || H == 0 || check_large(z) != AJVP_OK) return 0;
    const uint64_t least = host::stats_bytes(B * H, Lq) + range_bytes(B, Lk);
    int dev = 0;
    if (host::device(&dev) != AJVP_OK) return least;  // no usable device: the minimum
    return least + 2u * host::partial_bytes(B * Hkv, Lk, split_parts(z, host::sm_count(dev)));
}

int attn_jvp_bwd_scored(const void *q, const void *k, const void *v, const void *tq, const void *tk, const void *tv,
                        const void *o, const void *to, const float *lse, const float *mu, const void *dout,
                        const void *dtout, void *dq, void *dk, void *dv, void *dtq, void *dtk, void *dtv,
                        const float *slopes, const int32_t *key_begin, const int32_t *key_end, int64_t B, int64_t H,
                        int64_t Hkv, int64_t Lq, int64_t Lk, int64_t d, float scale, float softcap, void *workspace,
                        uint64_t workspace_bytes, void *stream) {
    const Sizes z{B, H, Hkv, Lq, Lk, d};
    int rc = check_sizes(z, scale, softcap);
    if (rc != AJVP_OK) return rc;
    if (B == 0 || Hkv == 0) return AJVP_OK;
    const cudaStream_t st = (cudaStream_t)stream;
    if ((rc = check_large(z)) != AJVP_OK) return rc;
    if (d != bwd::HD) return AJVP_ERR_UNSUPPORTED_DIM;
    if (Lq == 0 || H == 0) {  // no query rows: the key-side gradients are zero
        void *zero[4] = {dk, dv, dtk, dtv};
        for (void *p : zero)
            if (!p) return AJVP_ERR_INVALID_ARG;
        for (void *p : zero) {
            const cudaError_t e = cudaMemsetAsync(p, 0, (size_t)(B * Hkv * Lk * d) * 2u, st);
            if (e != cudaSuccess) return host::fail(e);
        }
        return AJVP_OK;
    }
    for (const void *p : {q, k, v, tq, tk, tv, o, to, (const void *)lse, (const void *)mu, dout, dtout,
                          (const void *)dq, (const void *)dk, (const void *)dv, (const void *)dtq, (const void *)dtk,
                          (const void *)dtv}) {
        if (!p) return AJVP_ERR_INVALID_ARG;
        if (!host::aligned(p, 16)) return AJVP_ERR_MISALIGNED;
    }
    for (const void *p : {(const void *)slopes, (const void *)key_begin, (const void *)key_end})
        if (!host::aligned(p, 4)) return AJVP_ERR_MISALIGNED;
    const int64_t BH = B * H, BHk = B * Hkv;
    const uint64_t stats = host::stats_bytes(BH, Lq), ranges = range_bytes(B, Lk);
    if (!workspace || !host::aligned(workspace, 256) || workspace_bytes < stats + ranges) return AJVP_ERR_WORKSPACE;
    int dev = 0;
    if ((rc = setup(&dev)) != AJVP_OK) return rc;
    if ((rc = host::encoder()) != AJVP_OK) return rc;
    // cut the streamed queries of the key side into parts when its key tiles alone
    // cannot fill the GPU and the workspace holds the partial sums
    int64_t parts = split_parts(z, host::sm_count(dev));
    const uint64_t part_bytes = host::partial_bytes(BHk, Lk, parts);
    if (workspace_bytes < stats + ranges + 2u * part_bytes) parts = 1;
    uint8_t *const ws = static_cast<uint8_t *>(workspace);
    float *const partial_k = reinterpret_cast<float *>(ws + stats + ranges);
    float *const partial_v = reinterpret_cast<float *>(ws + stats + ranges + part_bytes);

    const long long rows = (long long)(BH * Lq);
    const unsigned n_stats = (unsigned)std::min<long long>((rows + 7) / 8, 148LL * 16);
    const int64_t n_ranges = key_begin || key_end ? (Lk + 127) / 128 * B : 0;
    const Score bounds = make_score(z, scale, softcap, slopes, key_begin, key_end);
    Score score = bounds;
    int2 *const range_out = reinterpret_cast<int2 *>(ws + stats);
    if (n_ranges > 0) score.qrange = range_out;
    bwd::ParamsAll p;
    if ((rc = bwd_params(&p.k, {k, tk, v, tv}, {q, tq}, {dtout, dout}, dk, dtk, scale, score, workspace, BHk, BH, Lk, Lq,
                         Lq, scale, parts, partial_k)) != AJVP_OK)
        return rc;
    if ((rc = bwd_params(&p.q, {q, tq, dtout, dout}, {k, tk}, {v, tv}, dq, dtq, scale, score, workspace, BH, BHk, Lq, Lk,
                         Lq, scale, 1, nullptr)) != AJVP_OK)
        return rc;
    if ((rc = bwd_params(&p.v, {k, tk}, {dout, dtout}, {q, tq}, dv, dtv, 1.f, score, workspace, BHk, BH, Lk, Lq, Lq,
                         scale, parts, partial_v)) != AJVP_OK)
        return rc;
    const int64_t n_key = (int64_t)p.k.n_rtiles * BHk * parts, n_query = (int64_t)p.q.n_rtiles * BH;
    if (2 * n_key + n_query >= (int64_t(1) << 31)) return AJVP_ERR_TOO_LARGE;
    p.n_k = (unsigned)n_key;
    p.n_q = (unsigned)n_query;
    const auto *const ob = static_cast<const __nv_bfloat16 *>(o), *const tob = static_cast<const __nv_bfloat16 *>(to);
    const auto *const db = static_cast<const __nv_bfloat16 *>(dout);
    const auto *const dtb = static_cast<const __nv_bfloat16 *>(dtout);
    if (n_ranges > 0)
        bwd::scored_prep_kernel<<<n_stats + (unsigned)n_ranges, 256, 0, st>>>(ob, tob, db, dtb, lse, mu,
                                                                              static_cast<float4 *>(workspace), rows,
                                                                              (unsigned)n_ranges, bounds, (int)Lq,
                                                                              (int)Lk, range_out);
    else
        bwd::bwd_rowstats_kernel<<<n_stats, 256, 0, st>>>(ob, tob, db, dtb, lse, mu, static_cast<float4 *>(workspace),
                                                          rows);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host::fail(e);
    rc = with_mask(mask_bits(softcap, slopes), [&](auto mask) -> int {
        constexpr int M = decltype(mask)::value;
        const dim3 grid((unsigned)(2 * n_key + n_query));
        if (parts > 1)
            bwd::attn_jvp_bwd_scored_kernel<M, true><<<grid, bwd::NTHREADS, bwd::SMEM_ALL, st>>>(p);
        else
            bwd::attn_jvp_bwd_scored_kernel<M, false><<<grid, bwd::NTHREADS, bwd::SMEM_ALL, st>>>(p);
        const cudaError_t e1 = cudaGetLastError();
        return e1 == cudaSuccess ? AJVP_OK : host::fail(e1);
    });
    if (rc != AJVP_OK || parts <= 1) return rc;
    const long long krows = (long long)(BHk * Lk), n4 = krows * 2 * (bwd::HD / 4);
    bwd::scored_reduce_kernel<<<dim3((unsigned)std::min<long long>((n4 + 255) / 256, 148LL * 8), 2), 256, 0, st>>>(
        reinterpret_cast<const float4 *>(partial_k), reinterpret_cast<const float4 *>(partial_v), (int)parts, krows,
        static_cast<__nv_bfloat16 *>(dk), static_cast<__nv_bfloat16 *>(dtk), static_cast<__nv_bfloat16 *>(dv),
        static_cast<__nv_bfloat16 *>(dtv), scale);
    e = cudaGetLastError();
    return e == cudaSuccess ? AJVP_OK : host::fail(e);
}

}  // extern "C"
