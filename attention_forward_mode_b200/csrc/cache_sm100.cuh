// cache_sm100.cuh -- the paged 8-bit key/value cache: appending rotated keys
// and values, and attention + JVP of a few query tokens per sequence over it.
//
// A page holds `page` tokens of every key head: codes [pages][Hkv][page][128]
// in e4m3 and one scale [pages][Hkv] each for keys and values; value = code x
// scale.  Scales are powers of two, the smallest that brings the page's largest
// value to at most 448, so dividing by a scale is exact, and so is rescaling a
// page's codes when a later token needs a larger scale (but for codes that
// become subnormal).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "score_sm100.cuh"

namespace ajvp {
namespace cache {

constexpr int HD = 128;
constexpr int SCALE_MIN = -100, SCALE_MAX = 100;  // exponents of the scales

// exponent of the smallest power of two s with amax <= 448 s (448 = 1.75 2^8)
__device__ __forceinline__ int scale_exponent(float amax) {
    if (!(amax > 0.f)) return SCALE_MIN;
    const uint32_t bits = __float_as_uint(amax);
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, SCALE_MIN), SCALE_MAX);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 .. 127
// exponent of a scale written by the append kernel
__device__ __forceinline__ int exponent_of(float scale) {
    return min(max((int)((__float_as_uint(scale) >> 23) & 255u) - 127, SCALE_MIN), SCALE_MAX);
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float4 x) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x.x, x.y), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x.z, x.w), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
// two e4m3 codes (the low 16 bits) as f16x2; exact
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
__device__ __forceinline__ float4 unpack_e4m3x4(uint32_t w) {
    const uint32_t a = e4m3x2_to_f16x2(w & 0xffffu), b = e4m3x2_to_f16x2(w >> 16);
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
    return make_float4(x.x, x.y, y.x, y.y);
}

// ------------------------------------------------------------------ append
struct AppendParams {
    const __nv_bfloat16 *k, *v;    // [Hkv][total][128] new tokens, sequence b at rows cu[b] .. cu[b + 1] - 1
    const __nv_bfloat16 *q, *tq;   // [H][total][128] or NULL: rotated into q_out, tq_out
    __nv_bfloat16 *q_out, *tq_out;
    uint8_t *k8, *v8;
    float *ks, *vs;
    const int *table;              // [n_seq][table_width] page of each run of `page` tokens
    const int *lens;               // [n_seq] tokens already cached
    const int *cu;                 // [n_seq + 1]
    const float *cos, *sin;        // [n_pos][64] by token position, or NULL: no rotation
    int n_seq, H, Hkv, total, n_pages, page, table_width, n_pos, interleaved;
    int n_slots;                   // page CTAs per key head (an upper bound of the touched pages)
};

constexpr int APPEND_THREADS = 256, APPEND_WARPS = APPEND_THREADS / 32;
constexpr int ROWS_PER_CTA = 32;  // query rows per CTA

// Four channels of a row (lane l: 4l .. 4l + 3) turned by the angles of the
// row's position.  Products and sums are rounded one by one (no fused
// multiply-add), so that the result, and with it the scale, is that of the
// formula evaluated step by step in fp32.
__device__ __forceinline__ float4 rotate(const AppendParams &p, float4 x, int pos, int lane) {
    const size_t at = (size_t)min(max(pos, 0), p.n_pos - 1) * (HD / 2);
    if (p.interleaved) {  // pairs (4l, 4l + 1), (4l + 2, 4l + 3): angles 2l, 2l + 1
        const float2 c = *reinterpret_cast<const float2 *>(p.cos + at + 2 * lane);
        const float2 s = *reinterpret_cast<const float2 *>(p.sin + at + 2 * lane);
        return make_float4(__fsub_rn(__fmul_rn(x.x, c.x), __fmul_rn(x.y, s.x)),
                           __fadd_rn(__fmul_rn(x.y, c.x), __fmul_rn(x.x, s.x)),
                           __fsub_rn(__fmul_rn(x.z, c.y), __fmul_rn(x.w, s.y)),
                           __fadd_rn(__fmul_rn(x.w, c.y), __fmul_rn(x.z, s.y)));
    }
    // pairs (i, i + 64): lane l's partner channels are lane l ^ 16's
    const float4 c = *reinterpret_cast<const float4 *>(p.cos + at + 4 * (lane & 15));
    const float4 s = *reinterpret_cast<const float4 *>(p.sin + at + 4 * (lane & 15));
    const float4 y = make_float4(__shfl_xor_sync(0xffffffffu, x.x, 16), __shfl_xor_sync(0xffffffffu, x.y, 16),
                                 __shfl_xor_sync(0xffffffffu, x.z, 16), __shfl_xor_sync(0xffffffffu, x.w, 16));
    const float sign = lane < 16 ? -1.f : 1.f;  // first halves a cos - b sin, second halves b cos + a sin
    return make_float4(__fadd_rn(__fmul_rn(x.x, c.x), sign * __fmul_rn(y.x, s.x)),
                       __fadd_rn(__fmul_rn(x.y, c.y), sign * __fmul_rn(y.y, s.y)),
                       __fadd_rn(__fmul_rn(x.z, c.z), sign * __fmul_rn(y.z, s.z)),
                       __fadd_rn(__fmul_rn(x.w, c.w), sign * __fmul_rn(y.w, s.w)));
}

__device__ __forceinline__ float4 load_bf16x4(const __nv_bfloat16 *row, int lane) {
    const uint2 u = *reinterpret_cast<const uint2 *>(row + 4 * lane);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float amax4(float m, float4 x) {
    return fmaxf(fmaxf(m, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
}

// rows cu[b] .. of sequence b, clamped into the packed tensors so that bad offsets stay memory-safe
__device__ __forceinline__ int2 new_rows(const AppendParams &p, int b) {
    const int r0 = min(max(p.cu[b], 0), p.total);
    return make_int2(r0, max(min(max(p.cu[b + 1], 0), p.total), r0));
}

// One CTA per (touched page, key head), both caches: the new tokens' largest
// value (rotated keys), the page's new scale, codes of its earlier tokens moved
// to that scale when it grew, then the new codes.  The page is one CTA's own, so
// nothing is atomic.  CTAs past the page slots rotate q and tq, ROWS_PER_CTA
// rows of a head each.  Bound by its bytes (keys and values read twice, the
// second time from L1/L2).
static __global__ void __launch_bounds__(APPEND_THREADS) cache_append_kernel(const __grid_constant__ AppendParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_page_ctas = p.n_slots * p.Hkv;
    if ((int)blockIdx.x >= n_page_ctas) {
        const int chunks = (p.total + ROWS_PER_CTA - 1) / ROWS_PER_CTA;
        const int u = (int)blockIdx.x - n_page_ctas, h = u / chunks, row0 = (u - h * chunks) * ROWS_PER_CTA;
        for (int row = row0 + warp; row < min(row0 + ROWS_PER_CTA, p.total); row += APPEND_WARPS) {
            int lo = 0, hi = p.n_seq;  // the last sequence that starts at or before the row
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (p.cu[mid] <= row) lo = mid; else hi = mid;
            }
            const int2 rows = new_rows(p, lo);
            if (row < rows.x || row >= rows.y) continue;  // behind the last sequence: not written
            const int pos = max(p.lens[lo], 0) + row - rows.x;
            const size_t off = ((size_t)h * p.total + row) * HD;
            const float4 x = rotate(p, load_bf16x4(p.q + off, lane), pos, lane);
            uint2 w = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
            *reinterpret_cast<uint2 *>(p.q_out + off + 4 * lane) = w;
            if (p.tq) {
                const float4 t = rotate(p, load_bf16x4(p.tq + off, lane), pos, lane);
                w = make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
                *reinterpret_cast<uint2 *>(p.tq_out + off + 4 * lane) = w;
            }
        }
        return;
    }
    // the slot'th touched page over all sequences, counted by every warp for itself
    const int slot = (int)blockIdx.x / p.Hkv, hk = (int)blockIdx.x - slot * p.Hkv;
    int before = 0, b = -1, nth = 0;
    for (int b0 = 0; b0 < p.n_seq && b < 0; b0 += 32) {
        int pages = 0;
        if (b0 + lane < p.n_seq) {
            const int2 rows = new_rows(p, b0 + lane);
            const int start = max(p.lens[b0 + lane], 0), n = rows.y - rows.x;
            pages = n > 0 ? (int)(((long long)start + n - 1) / p.page - start / p.page) + 1 : 0;
        }
        int upto = pages;  // inclusive sum over the lanes
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += x;
        }
        const unsigned own = __ballot_sync(0xffffffffu, slot >= before + upto - pages && slot < before + upto);
        if (own != 0u) {
            const int l = __ffs(own) - 1;
            b = b0 + l;
            nth = slot - before - __shfl_sync(0xffffffffu, upto - pages, l);
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (b < 0) return;  // past the last touched page (the same for the whole CTA)
    const int2 rows = new_rows(p, b);
    const int start = max(p.lens[b], 0), at = start / p.page + nth;
    if (at >= p.table_width) return;  // past the sequence's pages: not written
    const int id = p.table[(size_t)b * p.table_width + at];
    if (id < 0 || id >= p.n_pages) return;
    // tokens [kept, last) of the page are new: packed rows first, first + 1, ...
    const long long page0 = (long long)at * p.page;
    const int kept = (int)max((long long)start - page0, 0LL);
    const int last = (int)min((long long)start + (rows.y - rows.x) - page0, (long long)p.page);
    const int first = rows.x + (int)(page0 + kept - start);
    const __nv_bfloat16 *const krow = p.k + ((size_t)hk * p.total + first) * HD;
    const __nv_bfloat16 *const vrow = p.v + ((size_t)hk * p.total + first) * HD;
    const bool turn = p.cos != nullptr;

    float ka = 0.f, va = 0.f;
    for (int t = kept + warp; t < last; t += APPEND_WARPS) {
        float4 x = load_bf16x4(krow + (size_t)(t - kept) * HD, lane);
        if (turn) x = rotate(p, x, (int)(page0 + t), lane);
        ka = amax4(ka, x);
        va = amax4(va, load_bf16x4(vrow + (size_t)(t - kept) * HD, lane));
    }
    // positive floats order like their bits
    const uint32_t kb = __reduce_max_sync(0xffffffffu, __float_as_uint(ka));
    const uint32_t vb = __reduce_max_sync(0xffffffffu, __float_as_uint(va));
    __shared__ uint32_t s_k[APPEND_WARPS], s_v[APPEND_WARPS];
    if (lane == 0) {
        s_k[warp] = kb;
        s_v[warp] = vb;
    }
    const size_t sc = (size_t)id * p.Hkv + hk;
    // the old scales, read before any thread writes the new ones; a page that starts here has none
    const int ek_old = kept > 0 ? exponent_of(p.ks[sc]) : SCALE_MIN, ev_old = kept > 0 ? exponent_of(p.vs[sc]) : SCALE_MIN;
    __syncthreads();
    uint32_t km = s_k[0], vm = s_v[0];
#pragma unroll
    for (int w = 1; w < APPEND_WARPS; ++w) {
        km = max(km, s_k[w]);
        vm = max(vm, s_v[w]);
    }
    const int ek = max(scale_exponent(__uint_as_float(km)), ek_old), ev = max(scale_exponent(__uint_as_float(vm)), ev_old);
    if (threadIdx.x == 0) {
        p.ks[sc] = pow2(ek);
        p.vs[sc] = pow2(ev);
    }
    uint8_t *const kc = p.k8 + sc * p.page * HD, *const vc = p.v8 + sc * p.page * HD;
    auto moved = [&](uint8_t *codes, int from, int to) {
        const float r = from - to >= -126 ? pow2(from - to) : 0.f;
        for (int t = warp; t < kept; t += APPEND_WARPS) {
            uint32_t *const w = reinterpret_cast<uint32_t *>(codes + (size_t)t * HD) + lane;
            const float4 x = unpack_e4m3x4(*w);
            *w = pack_e4m3x4(make_float4(x.x * r, x.y * r, x.z * r, x.w * r));
        }
    };
    if (kept > 0 && ek > ek_old) moved(kc, ek_old, ek);
    if (kept > 0 && ev > ev_old) moved(vc, ev_old, ev);
    const float kr = pow2(-ek), vr = pow2(-ev);
    for (int t = kept + warp; t < last; t += APPEND_WARPS) {
        float4 x = load_bf16x4(krow + (size_t)(t - kept) * HD, lane);
        if (turn) x = rotate(p, x, (int)(page0 + t), lane);
        reinterpret_cast<uint32_t *>(kc + (size_t)t * HD)[lane] =
            pack_e4m3x4(make_float4(x.x * kr, x.y * kr, x.z * kr, x.w * kr));
        const float4 y = load_bf16x4(vrow + (size_t)(t - kept) * HD, lane);
        reinterpret_cast<uint32_t *>(vc + (size_t)t * HD)[lane] =
            pack_e4m3x4(make_float4(y.x * vr, y.y * vr, y.z * vr, y.w * vr));
    }
}

// --------------------------------------------------------------- attention
// O, tO of n query tokens per sequence over the cache.  The rows of one key
// head (its group's heads x n tokens) are the M rows of m16n8k16 products:
// with a tangent, rows 0-7 of a tile are queries and rows 8-15 their tangents,
// so one thread holds S and dS of the same (row, key), and the second product
// of [P ; P dS] with V gives O and T = sum p dS V at once.  The cache carries
// no tangent, so tO = T / l - mu O.
//
// This is a decoding step: the work is to read the codes once.  So warps take
// runs of 16 tokens each, copy them ahead through rings of their own in shared
// memory (every lane reads back only what it copied), and turn codes into f16
// operands in registers: 16-byte pieces of key rows are B fragments of Q K^T
// (the order of channels inside a product is free, and the query fragments
// follow it), and bytes of value rows of two tokens pair up as B fragments of
// P V.  mma.sync rather than tcgen05: the products of 16 rows are a few percent
// of the time, and 128-row accumulators in tensor memory would be empty but for
// those rows.  Splits of a sequence are the CTAs of one cluster, which join
// their sums through distributed shared memory: no workspace, one launch, and a
// fixed order of additions.
//
// f16 operands: queries and tangents are scaled by a power of two per row to at
// most 2 (bf16 values are then exact but for those 2^-14 below the row's
// largest); P is weighted by its page's value scale, and the running reference
// M covers both, so |P| <= 2^8; dS is taken relative to the largest key scale
// so far (E) and 2^-10, so that |dS| < 2^7 and |P dS| < 2^15.
struct AttnParams {
    const __nv_bfloat16 *q, *tq;  // row (b, h, t) at q_b b + q_h h + q_t t channels; packed: cu[b] + t in place of t
    __nv_bfloat16 *o, *to;        // rows o_b b + o_h h + t (packed: + cu[b])
    float *lse;                   // one per output row, or NULL
    long long q_b, q_h, q_t, o_b, o_h;
    const int *cu;                // packed: [B + 1] starts of the sequences' rows, else NULL
    int total;                    // packed: rows of a head
    const uint8_t *k8, *v8;
    const float *ks, *vs;
    const int *table, *lens;
    const float *slopes;          // [H] or NULL
    float cap_in, cap_out;        // 2 / c (of scaled scores, in e-units) and c log2(e), 0: no cap
    float scale;
    int B, H, Hkv, group, n_pages, page, table_width, causal;
    int n;                        // query tokens per sequence (packed: of the longest)
    int tiles;                    // row tiles per (sequence, key head)
    int splits;                   // CTAs per cluster
};

constexpr int WARPS = 4, THREADS = WARPS * 32;
constexpr int STAGES = 4;
constexpr int STAGE_BYTES = 8 * 512;                 // 16 tokens of keys and values
constexpr int RING_BYTES = STAGES * STAGE_BYTES;     // per warp
constexpr int SCALES_OFF = WARPS * RING_BYTES;       // float2 per warp and stage
constexpr int STATS_OFF = SCALES_OFF + WARPS * STAGES * 8;
constexpr int TAN_UNITS = 49;
constexpr int STATS_FLOATS = TAN_UNITS + 8;          // m, l, g per row, E, the tangent rows' units
constexpr int ATTN_SMEM = STATS_OFF + (WARPS + 1) * 64 * 4;
static_assert(STATS_FLOATS <= 64 && 16 * HD * 4 <= RING_BYTES, "the sums of a warp fit its ring");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// kTan: 8 query rows and their tangents per tile, else 16 query rows.
template <bool kTan>
__global__ void __launch_bounds__(THREADS, 3) cache_attn_kernel(const __grid_constant__ AttnParams p) {
    constexpr int ROWS = kTan ? 8 : 16;    // query rows of a tile
    constexpr int R = kTan ? 1 : 2;        // query rows per thread
    extern __shared__ __align__(16) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gr = lane >> 2, c = lane & 3;  // fragment row and column group
    const int rank = (int)blockIdx.x % p.splits;
    const int unit = (int)blockIdx.x / p.splits;
    const int tile = unit % p.tiles, bh = unit / p.tiles;
    const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
    int n = p.n, first = 0;  // this sequence's query tokens and their first row
    if (p.cu) {
        first = min(max(p.cu[b], 0), p.total);
        n = min(max(min(max(p.cu[b + 1], 0), p.total) - first, 0), p.n);
    }
    const int n_rows = p.group * n;
    if (tile * ROWS >= n_rows) return;  // (the same for every CTA of the cluster)
    const int len = min(max(p.lens[b], 0), p.table_width * p.page);
    // this CTA's runs of 16 tokens
    const int runs = (len + 15) >> 4;
    const int per = (runs + p.splits - 1) / p.splits;
    const int run0 = min(rank * per, runs), run1 = min(run0 + per, runs);

    // query fragments: row gr (and gr + 8: its tangent, or query row gr + 8); product s
    // takes channels base(s) + {0, 1, 2, 3} of this lane, base = 16 c + 4 s, from s = 4 on
    // 64 + 16 c + 4 (s - 4)
    uint32_t aq[8][4];
    float row_scale[2] = {0.f, 0.f};  // power of two per row, times the softmax scale
    int end[R];                       // keys 0 .. end - 1 are visible
    int pos[R];
    float slope2[R];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = tile * ROWS + gr + (kTan ? 0 : 8 * i);
        const bool live = r < n_rows;
        const int h = live ? hk * p.group + r / n : 0, t = live ? r % n : 0;
        const __nv_bfloat16 *src = (kTan && i == 1 ? p.tq : p.q) + (p.q_b * b + p.q_h * h + p.q_t * (first + t));
        uint2 raw[8];
        float amax = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            raw[s] = live ? *reinterpret_cast<const uint2 *>(src + (s >> 2) * 64 + 16 * c + 4 * (s & 3)) : make_uint2(0u, 0u);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint32_t u = w ? raw[s].y : raw[s].x;
                amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u << 16)), fabsf(__uint_as_float(u & 0xffff0000u))));
            }
        }
        amax = quad_max(amax);
        // 2^e with amax in [2^e, 2^(e + 1))
        const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -120), 120);
        const float inv = pow2(-e);
        row_scale[i] = pow2(e) * p.scale;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            aq[s][i] = pack_f16x2(__uint_as_float(raw[s].x << 16) * inv, __uint_as_float(raw[s].x & 0xffff0000u) * inv);
            aq[s][2 + i] = pack_f16x2(__uint_as_float(raw[s].y << 16) * inv, __uint_as_float(raw[s].y & 0xffff0000u) * inv);
        }
        if (i < R) {
            pos[i] = len - n + t;
            end[i] = live && p.causal ? min(max(pos[i] + 1, 0), len) : len;
            slope2[i] = p.slopes && live ? p.slopes[h] * 1.4426950408889634f : 0.f;
        }
    }
    int least = end[0];  // keys that every row of the tile sees
#pragma unroll
    for (int i = 1; i < R; ++i) least = min(least, end[i]);
    least = __reduce_min_sync(0xffffffffu, least);

    float acc[16][4];
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    float m[R], l[R], g = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
    int E = SCALE_MIN;

    const uint32_t ring = sbase + (uint32_t)warp * RING_BYTES + (uint32_t)lane * 16u;
    const uint32_t scales = sbase + SCALES_OFF + (uint32_t)warp * STAGES * 8u;
    const int *const table = p.table + (size_t)b * p.table_width;
    auto page_of = [&](int run) -> int { return run < run1 ? table[run * 16 / p.page] : -1; };
    auto copy = [&](int run, int id, int stage) {
        if (run < run1 && id >= 0 && id < p.n_pages) {
            const size_t sc = (size_t)id * p.Hkv + hk;
            const size_t row0 = sc * p.page + (size_t)(run * 16 % p.page);
            const uint8_t *const kr = p.k8 + (row0 + gr) * HD + 16 * c;
            const uint8_t *const vr = p.v8 + (row0 + 2 * c) * HD + 16 * gr;
            const uint32_t d = ring + (uint32_t)stage * STAGE_BYTES;
            cp_async16(d, kr);
            cp_async16(d + 512, kr + 64);
            cp_async16(d + 1024, kr + 8 * HD);
            cp_async16(d + 1536, kr + 8 * HD + 64);
            cp_async16(d + 2048, vr);
            cp_async16(d + 2560, vr + HD);
            cp_async16(d + 3072, vr + 8 * HD);
            cp_async16(d + 3584, vr + 9 * HD);
            if (lane == 0) {
                cp_async4(scales + (uint32_t)stage * 8u, p.ks + sc);
                cp_async4(scales + (uint32_t)stage * 8u + 4u, p.vs + sc);
            }
        }
        cp_async_commit();
    };
    // ids of the pages of the runs in flight (the run being worked on first), and of the next one
    int ids[STAGES];
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) ids[s] = page_of(run0 + warp + s * WARPS);
    ids[STAGES - 1] = page_of(run0 + warp + (STAGES - 1) * WARPS);
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) copy(run0 + warp + s * WARPS, ids[s], s);
    int stage = 0;
    for (int run = run0 + warp; run < run1; run += WARPS) {
        const int id = ids[0];
        copy(run + (STAGES - 1) * WARPS, ids[STAGES - 1], (stage + STAGES - 1) % STAGES);
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) ids[s] = ids[s + 1];
        ids[STAGES - 1] = page_of(run + STAGES * WARPS);
        cp_async_wait<STAGES - 1>();
        __syncwarp();  // the scales are lane 0's copies
        const uint32_t d = ring + (uint32_t)stage * STAGE_BYTES;
        const uint32_t sc = scales + (uint32_t)stage * 8u;
        stage = (stage + 1) % STAGES;
        if (id < 0 || id >= p.n_pages) continue;  // no such page: its tokens are hidden
        float kscale, vscale;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(kscale), "=f"(vscale) : "r"(sc) : "memory");

        float S[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) S[nt][i] = 0.f;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint4 u = ld_shared_u4(d + (uint32_t)(nt * 2 + half) * 512u);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    mma_f16(S[nt], aq[half * 4 + s], e4m3x2_to_f16x2(w[s] & 0xffffu), e4m3x2_to_f16x2(w[s] >> 16));
            }
        }
        // scores in log2 units of keys run * 16 + 8 nt + 2 c + {0, 1}; row i of this thread
        // sits in S[nt][2 i], S[nt][2 i + 1] (kTan: dS in S[nt][2], S[nt][3])
        const bool all = (run + 1) * 16 <= least;
        const float kq = kscale * row_scale[0];
        float y[R][4], dS[4];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float sc_i = (kTan ? kq : kscale * row_scale[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = run * 16 + 8 * (e >> 1) + 2 * c + (e & 1);
                const float z = S[e >> 1][2 * i + (e & 1)] * sc_i;
                if constexpr (kTan) dS[e] = S[e >> 1][2 + (e & 1)];
                float v = z * 1.4426950408889634f;
                if (p.cap_out > 0.f) {
                    float2 t, df;
                    cap2(make_float2(z, z), p.cap_in, t, df);
                    v = t.x * p.cap_out;
                    if constexpr (kTan) dS[e] *= df.x;
                }
                v = fmaf(-slope2[i], fabsf((float)(pos[i] - key)), v);
                const bool seen = all || key < end[i];
                y[i][e] = seen ? v : -INFINITY;
                if (kTan && !seen) dS[e] = 0.f;  // (codes past the end may be NaN)
            }
        }
        // running references of y + log2(value scale), lazily raised
        const int ev = exponent_of(vscale), ek = exponent_of(kscale);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float top = quad_max(fmaxf(fmaxf(y[i][0], y[i][1]), fmaxf(y[i][2], y[i][3]))) + (float)ev;
            const bool need = top > m[i] + 8.f;
            if (__any_sync(0xffffffffu, need)) {
                const float alpha = need ? ex2_approx(m[i] - top) : 1.f;
                if (need) m[i] = top;
                l[i] *= alpha;
                if (kTan) g *= alpha;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    acc[j][2 * i] *= alpha;
                    acc[j][2 * i + 1] *= alpha;
                    if (kTan) {
                        acc[j][2] *= alpha;
                        acc[j][3] *= alpha;
                    }
                }
            }
        }
        if (kTan && ek > E) {  // a larger key scale: T moves to it
            const float r = ek - E <= 126 ? pow2(E - ek) : 0.f;
            E = ek;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                acc[j][2] *= r;
                acc[j][3] *= r;
            }
        }
        uint32_t ap[4];
        const float rel = kTan ? pow2(max(ek - E, -116) - 10) : 0.f;
        float w4[2][4];  // P x value scale: [row][key], or P and P dS
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float ref = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float pe = ex2_approx(y[i][e] - ref);
                l[i] += pe;
                w4[i][e] = pe * vscale;
                if constexpr (kTan) {
                    g = fmaf(pe, dS[e] * (kscale * row_scale[1]), g);
                    w4[1][e] = w4[0][e] * (dS[e] * rel);
                }
            }
        }
        ap[0] = pack_f16x2(w4[0][0], w4[0][1]);
        ap[1] = pack_f16x2(w4[1][0], w4[1][1]);
        ap[2] = pack_f16x2(w4[0][2], w4[0][3]);
        ap[3] = pack_f16x2(w4[1][2], w4[1][3]);
        // values of tokens 2c, 2c + 1, 2c + 8, 2c + 9, channels 16 gr + j; tokens past the
        // end may hold anything (also NaN codes) and are zeroed
        uint4 v0 = ld_shared_u4(d + 2048u), v1 = ld_shared_u4(d + 2560u);
        uint4 v2 = ld_shared_u4(d + 3072u), v3 = ld_shared_u4(d + 3584u);
        if ((run + 1) * 16 > len) {
            const int left = len - run * 16 - 2 * c;
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            if (left <= 0) v0 = zero;
            if (left <= 1) v1 = zero;
            if (left <= 8) v2 = zero;
            if (left <= 9) v3 = zero;
        }
        const uint32_t a0[4] = {v0.x, v0.y, v0.z, v0.w}, a1[4] = {v1.x, v1.y, v1.z, v1.w};
        const uint32_t a2[4] = {v2.x, v2.y, v2.z, v2.w}, a3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t lo01 = __byte_perm(a0[w], a1[w], 0x5140), hi01 = __byte_perm(a0[w], a1[w], 0x7362);
            const uint32_t lo89 = __byte_perm(a2[w], a3[w], 0x5140), hi89 = __byte_perm(a2[w], a3[w], 0x7362);
            mma_f16(acc[4 * w], ap, e4m3x2_to_f16x2(lo01 & 0xffffu), e4m3x2_to_f16x2(lo89 & 0xffffu));
            mma_f16(acc[4 * w + 1], ap, e4m3x2_to_f16x2(lo01 >> 16), e4m3x2_to_f16x2(lo89 >> 16));
            mma_f16(acc[4 * w + 2], ap, e4m3x2_to_f16x2(hi01 & 0xffffu), e4m3x2_to_f16x2(hi89 & 0xffffu));
            mma_f16(acc[4 * w + 3], ap, e4m3x2_to_f16x2(hi01 >> 16), e4m3x2_to_f16x2(hi89 >> 16));
        }
    }
    cp_async_wait<0>();
    __syncwarp();

    // each warp's sums into its ring: [16 rows][128] (rows 8-15: T, or query rows 8-15), its
    // statistics beside them.  acc[j][0, 1] are row gr, channels 16 (2 c) + j and 16 (2 c + 1) + j.
    float *const mine = reinterpret_cast<float *>(smem + warp * RING_BYTES);
    float *const stats = reinterpret_cast<float *>(smem + STATS_OFF) + warp * 64;
#pragma unroll
    for (int i = 0; i < R; ++i) l[i] = quad_sum(l[i]);
    g = quad_sum(g);
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                *reinterpret_cast<float4 *>(mine + (gr + 8 * half) * HD + 32 * c + 16 * k + j) =
                    make_float4(acc[j][2 * half + k], acc[j + 1][2 * half + k], acc[j + 2][2 * half + k],
                                acc[j + 3][2 * half + k]);
    if (c == 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            stats[gr + 8 * i] = m[i];
            stats[16 + gr + 8 * i] = l[i];
        }
        if (kTan) stats[32 + gr] = g;
        if (kTan && warp == 0)  // the tangent rows' units, for this CTA's outputs
            (reinterpret_cast<float *>(smem + STATS_OFF) + WARPS * 64)[TAN_UNITS + gr] = row_scale[1];
        if (lane == 0) reinterpret_cast<int *>(stats)[48] = E;
    }
    __syncthreads();
    // the CTA's sums, in warp order, into warp 0's ring; statistics into slot WARPS
    const float *const st = reinterpret_cast<const float *>(smem + STATS_OFF);
    float *const cst = reinterpret_cast<float *>(smem + STATS_OFF) + WARPS * 64;
    int Ec = SCALE_MIN;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) Ec = max(Ec, reinterpret_cast<const int *>(st + 64 * w)[48]);
    auto weight = [](float m, float top) -> float { return m == -INFINITY ? 0.f : ex2_approx(m - top); };
    auto shrink = [](int e, int top) -> float { return e - top >= -126 ? pow2(e - top) : 0.f; };
    for (int x = threadIdx.x; x < 16 * HD / 4; x += THREADS) {
        const int r = x / (HD / 4);
        const int row = kTan ? (r & 7) : r;
        float top = st[row];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) top = fmaxf(top, st[64 * w + row]);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        float lt = 0.f, gt = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float a = weight(st[64 * w + row], top);
            lt = fmaf(a, st[64 * w + 16 + row], lt);
            if (kTan) gt = fmaf(a, st[64 * w + 32 + row], gt);
            const float f = kTan && r >= 8 ? a * shrink(reinterpret_cast<const int *>(st + 64 * w)[48], Ec) : a;
            const float4 v = *reinterpret_cast<const float4 *>(smem + w * RING_BYTES + x * 16);
            sum.x = fmaf(f, v.x, sum.x);
            sum.y = fmaf(f, v.y, sum.y);
            sum.z = fmaf(f, v.z, sum.z);
            sum.w = fmaf(f, v.w, sum.w);
        }
        *reinterpret_cast<float4 *>(smem + x * 16) = sum;  // (this thread's own place in warp 0's ring)
        if ((x & (HD / 4 - 1)) == 0 && r == row) {
            cst[row] = top;
            cst[16 + row] = lt;
            if (kTan) cst[32 + row] = gt;
        }
        if (x == 0) reinterpret_cast<int *>(cst)[48] = Ec;
    }
    auto cluster_sync = [&]() {
        if (p.splits > 1)
            asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        else
            __syncthreads();
    };
    cluster_sync();
    // the cluster's sums, in rank order: the ranks share out the tile's rows x channels
    const uint32_t cstat = sbase + STATS_OFF + WARPS * 256u;
    for (int x = rank * THREADS + (int)threadIdx.x; x < ROWS * HD / 4; x += p.splits * THREADS) {
        const int row = x / (HD / 4), d4 = x % (HD / 4), r = tile * ROWS + row;
        if (r >= n_rows) continue;
        float top = -INFINITY;
        int Et = SCALE_MIN;
        for (int s = 0; s < p.splits; ++s) {
            const uint32_t a = cluster_map(cstat, (uint32_t)s);
            top = fmaxf(top, ld_cluster(a + 4u * row));
            Et = max(Et, __float_as_int(ld_cluster(a + 4u * 48)));
        }
        float4 so = make_float4(0.f, 0.f, 0.f, 0.f), sT = so;
        float lt = 0.f, gt = 0.f;
        for (int s = 0; s < p.splits; ++s) {
            const uint32_t a = cluster_map(cstat, (uint32_t)s), v = cluster_map(sbase, (uint32_t)s);
            const float f = weight(ld_cluster(a + 4u * row), top);
            lt = fmaf(f, ld_cluster(a + 4u * (16 + row)), lt);
            const float4 o4 = ld_cluster4(v + (uint32_t)(row * HD + 4 * d4) * 4u);
            so.x = fmaf(f, o4.x, so.x);
            so.y = fmaf(f, o4.y, so.y);
            so.z = fmaf(f, o4.z, so.z);
            so.w = fmaf(f, o4.w, so.w);
            if constexpr (kTan) {
                gt = fmaf(f, ld_cluster(a + 4u * (32 + row)), gt);
                const float ft = f * shrink(__float_as_int(ld_cluster(a + 4u * 48)), Et);
                const float4 t4 = ld_cluster4(v + (uint32_t)((row + 8) * HD + 4 * d4) * 4u);
                sT.x = fmaf(ft, t4.x, sT.x);
                sT.y = fmaf(ft, t4.y, sT.y);
                sT.z = fmaf(ft, t4.z, sT.z);
                sT.w = fmaf(ft, t4.w, sT.w);
            }
        }
        const float inv = lt > 0.f ? 1.f / lt : 0.f;  // a row that sees no key: zeros, lse = -infinity
        const float4 ov = make_float4(so.x * inv, so.y * inv, so.z * inv, so.w * inv);
        const int h = hk * p.group + r / n, t = r % n;
        const size_t out = (size_t)(p.o_b * b + p.o_h * h + first + t);
        *reinterpret_cast<uint2 *>(p.o + out * HD + 4 * d4) = make_uint2(pack_bf16x2(ov.x, ov.y), pack_bf16x2(ov.z, ov.w));
        if constexpr (kTan) {
            // T is in units of 2^(E + 10) times the tangent row's
            const float mu = gt * inv;
            const float unit = cst[TAN_UNITS + row] * pow2(Et) * (1024.f * inv);
            *reinterpret_cast<uint2 *>(p.to + out * HD + 4 * d4) =
                make_uint2(pack_bf16x2(fmaf(-mu, ov.x, sT.x * unit), fmaf(-mu, ov.y, sT.y * unit)),
                           pack_bf16x2(fmaf(-mu, ov.z, sT.z * unit), fmaf(-mu, ov.w, sT.w * unit)));
        }
        if (d4 == 0 && p.lse)
            p.lse[out] = lt > 0.f ? (top + __log2f(lt)) * 0.69314718055994531f : -INFINITY;
    }
    cluster_sync();  // no CTA leaves while another still reads its sums
}

}  // namespace cache
}  // namespace ajvp
