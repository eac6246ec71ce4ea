// cache.cu -- host side of the paged 8-bit cache: attn_jvp_cache_append and
// attn_jvp_fwd_cache.  Argument checks and launches; no device memory is
// allocated here.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "attn_jvp.h"
#include "cache_sm100.cuh"
#include "host_common.h"
#include "selftest_sm100.cuh"

using namespace ajvp;

namespace {

struct Setup {
    std::once_flag once;
    cudaError_t error = cudaSuccess;
};
Setup g_setup[host::kMaxDevices];

template <bool kTan, int NT, int W, int S>
cudaError_t set_attn() {
    cudaError_t e = cudaFuncSetAttribute(cache::cache_attn_kernel<kTan, NT, W, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         cache::attn_smem(W, S));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(cache::cache_attn_kernel<kTan, NT, W, S>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
}

int setup(int *dev) {
    int rc = host::device(dev);
    if (rc != AJVP_OK) return rc;
    Setup &s = g_setup[*dev];
    std::call_once(s.once, [&]() {
        for (cudaError_t e : {set_attn<true, 1, 4, 2>(), set_attn<true, 2, 4, 2>(), set_attn<false, 1, 4, 2>(),
                              set_attn<false, 2, 4, 2>(), set_attn<true, 1, 8, 3>(), set_attn<false, 1, 8, 3>()})
            if (s.error == cudaSuccess) s.error = e;
    });
    return s.error == cudaSuccess ? AJVP_OK : host::fail(s.error);
}

constexpr int64_t kMaxInt = int64_t(1) << 31;

// the cache's own sizes: page a multiple of 16, page indices and positions in 32 bits
int check_cache(int64_t n_seq, int64_t H, int64_t Hkv, int64_t n_pages, int64_t page, int64_t table_width, int64_t d) {
    if (n_seq < 0 || H < 0 || Hkv < 1 || H % Hkv != 0 || n_pages < 0 || page < 16 || page % 16 != 0 || table_width < 1 ||
        d < 1)
        return AJVP_ERR_INVALID_ARG;
    if (d != cache::HD) return AJVP_ERR_UNSUPPORTED_DIM;
    if (n_seq >= kMaxInt || H >= kMaxInt || n_pages >= kMaxInt || page > (1 << 16) || table_width >= (1 << 24) ||
        table_width * page >= (1 << 24) || Hkv >= kMaxInt / page || n_pages >= kMaxInt / (Hkv * page))
        return AJVP_ERR_TOO_LARGE;
    return AJVP_OK;
}

// How a launch is cut up.  A unit is a (sequence, key head, row tile); every
// further row tile of a key head reads its codes again (from L2).
struct Plan {
    int tiles;   // row tiles per (sequence, key head)
    int nt;      // column tiles of a row tile: 4 nt rows with tangents, 8 nt without
    int warps;   // per CTA
    int splits;  // CTAs per unit
    bool parts;  // they leave their sums in the workspace (else they are one cluster)
};

uint64_t plan_bytes(const Plan &p, int64_t n_seq, int64_t Hkv) {
    return p.parts ? (uint64_t)(n_seq * Hkv) * (uint64_t)p.tiles * (uint64_t)p.splits * cache::part_floats(p.nt) * 4u : 0u;
}

// Time of a plan in microseconds, within about 15 % over 18 shapes on a 148-SM B200:
// a fixed part, and the runs of 32 tokens of a warp at the latency of one, or those
// of an SM at its rate.
double plan_time(const Plan &p, int64_t units, int64_t runs, int sm_count) {
    const double ctas = (double)((units * p.splits + sm_count - 1) / sm_count);  // of an SM
    const double of_warp = (double)runs / (p.splits * p.warps);
    const double latency = p.nt == 1 ? 1.25 : 1.5, rate = p.nt == 1 ? 0.17 : 0.24;
    return (p.parts ? 8.5 : 7.0) + of_warp * std::max(latency, ctas * p.warps * rate);
}

// Without a workspace, or where it does not pay, the CTAs of a unit are a cluster.
// Measured over 18 shapes of 1 .. 64 sequences of 16 .. 32760 tokens, within 10 % of
// the best of all (nt, warps, splits) on a 148-SM B200 wherever the table is as long
// as the sequences:
// nt 2 (rows that do not fit one column tile): halves the reading and converting
//   of codes, but with few units two tiles run side by side (4 sequences, 4 key heads,
//   8 rows with tangents: 18 against 22 us; 16 sequences of 8 key heads, 5 rows: 92
//   against 62), so from 64 units on.
// splits: as many as keep every CTA resident at once (three of four warps per SM, two
//   of nt 2, a tenth left free for clusters that do not fill their place, a quarter by
//   clusters of 16), while each warp keeps two runs of 32 tokens (8 sequences of 2048,
//   12 heads: 1, 2, 4, 8 parts take 21, 15.5, 13, 21 us).
// warps 8: up to an SM's worth of CTAs, where only more warps per SM hide the
//   latency of a run (one sequence of 4096, 12 heads: 10.5 against 11.8 us); clusters of
//   them fill no more than some 120 SMs.
//
// With a workspace the CTAs of a unit may be any number anywhere.  Long contexts of
// few sequences then fill the GPU (one sequence of 32760 tokens, 40 heads on 8 key
// heads, with tangents: 24 against 35 us; 12 heads without: 21 against 28; of 200000
// tokens, one head: 37 against 73), while short ones gain a microsecond or two of
// kernel time and lose as much to the second launch, so from a modelled gain of
// an eighth on.
Plan make_plan(int64_t n_seq, int64_t Hkv, int64_t rows, bool tangent, int64_t tokens, int sm_count, bool workspace) {
    const int64_t one = tangent ? 4 : 8, runs = (tokens + 31) / 32;
    const int64_t least = 8;  // runs of a CTA: one per warp of eight, two per warp of four
    const auto units_of = [&](int nt) -> int64_t { return n_seq * Hkv * ((rows + nt * one - 1) / (nt * one)); };
    Plan p;
    p.nt = rows > one && units_of(2) >= 64 ? 2 : 1;
    const int64_t units = units_of(p.nt);
    const int64_t most8 = sm_count * 13 / 16, slots = sm_count * (p.nt == 1 ? 3 : 2);
    p.warps = p.nt == 1 && units * 8 <= most8 ? 8 : 4;
    p.splits = 1;
    p.parts = false;
    const auto fits = [&](int64_t splits) -> bool {
        const int64_t most = p.warps == 8 ? most8 : splits < 16 ? slots * 9 / 10 : slots * 3 / 4;
        return units * splits <= most && runs >= least * splits;
    };
    while (p.splits < 16 && fits(p.splits * 2)) p.splits *= 2;
    if (workspace) {
        double best = plan_time(p, units, runs, sm_count) * 0.875;
        for (int nt = 1; nt <= (rows > one ? 2 : 1); ++nt)
            for (int ctas = 1; ctas <= (nt == 1 ? 3 : 2); ++ctas) {  // of an SM
                Plan c;
                c.nt = nt;
                c.warps = 4;
                c.parts = true;
                const int64_t n = units_of(nt);
                c.splits = (int)std::min<int64_t>({ctas * sm_count / n, runs / least, cache::MOST_PARTS});
                if (c.splits < 2) continue;
                const double t = plan_time(c, n, runs, sm_count);
                if (t < best) {
                    best = t;
                    p = c;
                }
            }
    }
    p.tiles = (int)(units_of(p.nt) / (n_seq * Hkv));
    return p;
}

}  // namespace

namespace ajvp {
namespace host {
cudaError_t cache_selftest(uint64_t bound_ns, cudaStream_t stream) { return selftest_wait(bound_ns, false, stream); }
cudaError_t cache_status(int *word) {
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

int attn_jvp_cache_append(const void *k, const void *v, const void *q, const void *tq, void *q_out, void *tq_out,
                          void *k_cache, void *v_cache, float *k_scale, float *v_scale, const int32_t *block_table,
                          const int32_t *cache_lens, const int32_t *cu_seqlens, const float *cos, const float *sin,
                          int64_t n_seq, int64_t H, int64_t Hkv, int64_t total, int64_t n_pages, int64_t page,
                          int64_t table_width, int64_t n_pos, int64_t d, int interleaved, void *stream) {
    int rc = check_cache(n_seq, H, Hkv, n_pages, page, table_width, d);
    if (rc != AJVP_OK) return rc;
    if (total < 0 || n_pos < 0 || (!cos) != (!sin) || (cos && n_pos < 1)) return AJVP_ERR_INVALID_ARG;
    if ((q || tq) && !cos) return AJVP_ERR_INVALID_ARG;  // queries take part only to be rotated
    if ((tq && !q) || (!q) != (!q_out) || (!tq) != (!tq_out)) return AJVP_ERR_INVALID_ARG;
    if (total >= kMaxInt || n_pos >= kMaxInt) return AJVP_ERR_TOO_LARGE;
    if (n_seq == 0 || total == 0) return AJVP_OK;
    for (const void *p : {k, v, (const void *)k_cache, (const void *)v_cache, (const void *)k_scale,
                          (const void *)v_scale, (const void *)block_table, (const void *)cache_lens,
                          (const void *)cu_seqlens})
        if (!p) return AJVP_ERR_INVALID_ARG;
    for (const void *p : {k, v, q, tq, (const void *)q_out, (const void *)tq_out, (const void *)k_cache,
                          (const void *)v_cache, (const void *)cos, (const void *)sin})
        if (!host::aligned(p, 16)) return AJVP_ERR_MISALIGNED;
    for (const void *p : {(const void *)k_scale, (const void *)v_scale, (const void *)block_table,
                          (const void *)cache_lens, (const void *)cu_seqlens})
        if (!host::aligned(p, 4)) return AJVP_ERR_MISALIGNED;
    const int64_t slots = total / page + 2 * std::min(n_seq, total);  // a sequence's first and last pages may be partial
    const int64_t chunks = (total + cache::APPEND_WARPS - 1) / cache::APPEND_WARPS;
    // a warp per (page, head) while the sequences bring no more tokens on average than a warp holds
    const bool by_warp = total <= cache::HELD * n_seq;
    const int64_t page_ctas = by_warp ? (slots * Hkv + cache::APPEND_WARPS - 1) / cache::APPEND_WARPS : slots * Hkv;
    const int64_t grid = page_ctas + (q ? chunks * ((H + cache::HEADS_PER_WARP - 1) / cache::HEADS_PER_WARP) : 0);
    if (slots * Hkv >= kMaxInt) return AJVP_ERR_TOO_LARGE;
    if (grid >= kMaxInt) return AJVP_ERR_TOO_LARGE;
    int dev = 0;
    if ((rc = setup(&dev)) != AJVP_OK) return rc;
    cache::AppendParams p;
    std::memset(&p, 0, sizeof(p));
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.tq = static_cast<const __nv_bfloat16 *>(tq);
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.tq_out = static_cast<__nv_bfloat16 *>(tq_out);
    p.k8 = static_cast<uint8_t *>(k_cache);
    p.v8 = static_cast<uint8_t *>(v_cache);
    p.ks = k_scale;
    p.vs = v_scale;
    p.table = block_table;
    p.lens = cache_lens;
    p.cu = cu_seqlens;
    p.cos = cos;
    p.sin = sin;
    p.n_seq = (int)n_seq;
    p.H = (int)H;
    p.Hkv = (int)Hkv;
    p.total = (int)total;
    p.n_pages = (int)n_pages;
    p.page = (int)page;
    p.table_width = (int)table_width;
    p.n_pos = (int)n_pos;
    p.n_slots = (int)slots;
    using namespace ajvp::cache;
    auto *const kernel = !cos ? (by_warp ? cache_append_kernel<true, ROT_NONE> : cache_append_kernel<false, ROT_NONE>)
                         : interleaved ? (by_warp ? cache_append_kernel<true, ROT_PAIRS> : cache_append_kernel<false, ROT_PAIRS>)
                                       : (by_warp ? cache_append_kernel<true, ROT_HALVES> : cache_append_kernel<false, ROT_HALVES>);
    kernel<<<(unsigned)grid, APPEND_THREADS, 0, (cudaStream_t)stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? AJVP_OK : host::fail(e);
}

uint64_t attn_jvp_fwd_cache_workspace_bytes(int64_t n_seq, int64_t H, int64_t Hkv, int64_t n, int64_t page,
                                            int64_t table_width, int tangent) {
    if (check_cache(n_seq, H, Hkv, 1, page, table_width, cache::HD) != AJVP_OK || n < 1 || n_seq < 1 || H < 1) return 0;
    if (n >= kMaxInt || H / Hkv * n >= kMaxInt || n_seq * Hkv >= kMaxInt) return 0;
    int dev = 0;
    if (host::device(&dev) != AJVP_OK) return 0;
    return plan_bytes(make_plan(n_seq, Hkv, H / Hkv * n, tangent != 0, table_width * page, host::sm_count(dev), true),
                      n_seq, Hkv);
}

int attn_jvp_fwd_cache(const void *q, const void *tq, void *o, void *to, float *lse, const void *k_cache,
                       const void *v_cache, const float *k_scale, const float *v_scale, const int32_t *block_table,
                       const int32_t *cache_lens, const int32_t *cu_seqlens, const float *slopes, int64_t n_seq,
                       int64_t H, int64_t Hkv, int64_t n, int64_t total, int64_t stride_b, int64_t stride_h,
                       int64_t stride_t, int64_t n_pages, int64_t page, int64_t table_width, int64_t d, float scale,
                       float softcap, int causal, void *workspace, uint64_t workspace_bytes, void *stream) {
    int rc = check_cache(n_seq, H, Hkv, n_pages, page, table_width, d);
    if (rc != AJVP_OK) return rc;
    if (n < 0 || total < 0 || !std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f)
        return AJVP_ERR_INVALID_ARG;
    const float log2e = 1.4426950408889634f;
    if (softcap > 0.f && (!std::isfinite(2.f * log2e / softcap) || !std::isfinite(softcap * log2e)))
        return AJVP_ERR_INVALID_ARG;
    if (cu_seqlens && n > total) return AJVP_ERR_INVALID_ARG;
    if (n >= kMaxInt || total >= kMaxInt) return AJVP_ERR_TOO_LARGE;
    if (n_seq == 0 || H == 0 || n == 0 || (cu_seqlens && total == 0)) return AJVP_OK;
    for (const void *p : {q, (const void *)o, k_cache, v_cache, (const void *)k_scale, (const void *)v_scale,
                          (const void *)block_table, (const void *)cache_lens})
        if (!p) return AJVP_ERR_INVALID_ARG;
    if ((!tq) != (!to)) return AJVP_ERR_INVALID_ARG;
    for (const void *p : {q, tq, (const void *)o, (const void *)to, (const void *)lse, k_cache, v_cache})
        if (!host::aligned(p, 16)) return AJVP_ERR_MISALIGNED;
    if (stride_b % 8 != 0 || stride_h % 8 != 0 || stride_t % 8 != 0) return AJVP_ERR_MISALIGNED;
    for (const void *p : {(const void *)k_scale, (const void *)v_scale, (const void *)block_table,
                          (const void *)cache_lens, (const void *)cu_seqlens, (const void *)slopes})
        if (!host::aligned(p, 4)) return AJVP_ERR_MISALIGNED;
    if (!host::aligned(workspace, 256)) return AJVP_ERR_WORKSPACE;
    const int64_t group = H / Hkv;
    if (group * n >= kMaxInt || n_seq * Hkv >= kMaxInt) return AJVP_ERR_TOO_LARGE;
    if (n_pages < 1) return AJVP_ERR_INVALID_ARG;
    const int64_t most_tiles = (group * n + (tq ? 3 : 7)) / (tq ? 4 : 8);
    if (n_seq * Hkv >= kMaxInt / 16 / most_tiles) return AJVP_ERR_TOO_LARGE;
    int dev = 0;
    if ((rc = setup(&dev)) != AJVP_OK) return rc;
    if ((rc = host::encoder()) != AJVP_OK) return rc;
    cache::AttnParams p;
    std::memset(&p, 0, sizeof(p));
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.tq = static_cast<const __nv_bfloat16 *>(tq);
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.to = static_cast<__nv_bfloat16 *>(to);
    p.lse = lse;
    p.k8 = static_cast<const uint8_t *>(k_cache);
    p.v8 = static_cast<const uint8_t *>(v_cache);
    p.ks = k_scale;
    p.vs = v_scale;
    p.table = block_table;
    p.lens = cache_lens;
    p.slopes = slopes;
    p.cu = cu_seqlens;
    p.total = (int)total;
    p.q_b = cu_seqlens ? 0 : stride_b;
    p.q_h = stride_h;
    p.q_t = stride_t;
    p.o_b = cu_seqlens ? 0 : H * n;
    p.o_h = cu_seqlens ? total : n;
    p.cap_in = softcap > 0.f ? 2.f / softcap : 0.f;
    p.cap_w = softcap > 0.f ? 1.f / (softcap * log2e) : 0.f;
    p.cap_out = softcap * log2e;
    p.scale = scale;
    p.B = (int)n_seq;
    p.H = (int)H;
    p.Hkv = (int)Hkv;
    p.group = (int)group;
    p.n = (int)n;
    p.n_pages = (int)n_pages;
    p.page = (int)page;
    p.table_width = (int)table_width;
    p.causal = causal != 0;
    p.bound_ns = host::wait_bound_ns();
    if ((rc = host::encode_codes(&p.tm_k, k_cache, n_pages * Hkv * page, 16)) != AJVP_OK) return rc;
    if ((rc = host::encode_codes(&p.tm_v, v_cache, n_pages * Hkv * page, 16)) != AJVP_OK) return rc;
    p.page_magic = page == 16 ? 0u : (unsigned)(((uint64_t(1) << 32) + page / 16 - 1) / (page / 16));
    Plan plan = make_plan(n_seq, Hkv, group * n, tq != nullptr, table_width * page, host::sm_count(dev), true);
    if (plan.parts && (!workspace || workspace_bytes < plan_bytes(plan, n_seq, Hkv)))
        plan = make_plan(n_seq, Hkv, group * n, tq != nullptr, table_width * page, host::sm_count(dev), false);
    p.partial = plan.parts ? static_cast<float *>(workspace) : nullptr;
    p.tiles = plan.tiles;
    p.splits = plan.splits;

    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)(n_seq * Hkv * plan.tiles * plan.splits));
    cfg.blockDim = dim3(32 * plan.warps);
    cfg.dynamicSmemBytes = plan.warps == 4 ? cache::attn_smem(4, 2) : cache::attn_smem(8, 3);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = plan.parts ? 1u : (unsigned)p.splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e =
        plan.warps == 8 ? (tq ? cudaLaunchKernelEx(&cfg, cache::cache_attn_kernel<true, 1, 8, 3>, p)
                              : cudaLaunchKernelEx(&cfg, cache::cache_attn_kernel<false, 1, 8, 3>, p))
        : plan.nt == 1 ? (tq ? cudaLaunchKernelEx(&cfg, cache::cache_attn_kernel<true, 1, 4, 2>, p)
                             : cudaLaunchKernelEx(&cfg, cache::cache_attn_kernel<false, 1, 4, 2>, p))
                       : (tq ? cudaLaunchKernelEx(&cfg, cache::cache_attn_kernel<true, 2, 4, 2>, p)
                             : cudaLaunchKernelEx(&cfg, cache::cache_attn_kernel<false, 2, 4, 2>, p));
    if (e != cudaSuccess) return host::fail(e);
    if (!plan.parts) return AJVP_OK;
    cfg.gridDim = dim3((unsigned)(n_seq * Hkv * plan.tiles * plan.nt * (tq ? 4 : 8)));
    cfg.blockDim = dim3(32 * cache::JOIN_WARPS);
    cfg.dynamicSmemBytes = 0;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const cudaError_t e1 = plan.nt == 1 ? (tq ? cudaLaunchKernelEx(&cfg, cache::cache_join_kernel<true, 1>, p)
                                              : cudaLaunchKernelEx(&cfg, cache::cache_join_kernel<false, 1>, p))
                                        : (tq ? cudaLaunchKernelEx(&cfg, cache::cache_join_kernel<true, 2>, p)
                                              : cudaLaunchKernelEx(&cfg, cache::cache_join_kernel<false, 2>, p));
    return e1 == cudaSuccess ? AJVP_OK : host::fail(e1);
}

}  // extern "C"
