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

#include <type_traits>

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
    int n_seq, H, Hkv, total, n_pages, page, table_width, n_pos;
    int n_slots;                   // page CTAs per key head (an upper bound of the touched pages)
};

constexpr int APPEND_THREADS = 256, APPEND_WARPS = APPEND_THREADS / 32;
constexpr int HELD = 4;               // tokens of a page that a warp keeps in registers
constexpr int HEADS_PER_WARP = 4;     // query heads that share one reading of a row's angles

constexpr int ROT_NONE = 0, ROT_HALVES = 1, ROT_PAIRS = 2;
// The angles of a position for a lane's four channels (lane l: 4l .. 4l + 3).
struct Angles {
    float4 c, s;
};
template <int ROT>
__device__ __forceinline__ Angles angles_of(const AppendParams &p, int pos, int lane) {
    const size_t at = (size_t)min(max(pos, 0), p.n_pos - 1) * (HD / 2);
    Angles a;
    if constexpr (ROT == ROT_PAIRS) {  // pairs (4l, 4l + 1), (4l + 2, 4l + 3): angles 2l, 2l + 1
        const float2 c = *reinterpret_cast<const float2 *>(p.cos + at + 2 * lane);
        const float2 s = *reinterpret_cast<const float2 *>(p.sin + at + 2 * lane);
        a.c = make_float4(c.x, c.x, c.y, c.y);
        a.s = make_float4(-s.x, s.x, -s.y, s.y);
    } else {  // pairs (i, i + 64): lane l's partner channels are lane l ^ 16's
        a.c = *reinterpret_cast<const float4 *>(p.cos + at + 4 * (lane & 15));
        a.s = *reinterpret_cast<const float4 *>(p.sin + at + 4 * (lane & 15));
        if (lane < 16) a.s = make_float4(-a.s.x, -a.s.y, -a.s.z, -a.s.w);
    }
    return a;
}
// x cos + partner (-+ sin).  Products and sums are rounded one by one (no fused
// multiply-add), so that the result, and with it the scale, is that of the
// formula evaluated step by step in fp32.
template <int ROT>
__device__ __forceinline__ float4 rotate(float4 x, const Angles &a) {
    float4 y;
    if constexpr (ROT == ROT_PAIRS)
        y = make_float4(x.y, x.x, x.w, x.z);
    else
        y = make_float4(__shfl_xor_sync(0xffffffffu, x.x, 16), __shfl_xor_sync(0xffffffffu, x.y, 16),
                        __shfl_xor_sync(0xffffffffu, x.z, 16), __shfl_xor_sync(0xffffffffu, x.w, 16));
    return make_float4(__fadd_rn(__fmul_rn(x.x, a.c.x), __fmul_rn(y.x, a.s.x)),
                       __fadd_rn(__fmul_rn(x.y, a.c.y), __fmul_rn(y.y, a.s.y)),
                       __fadd_rn(__fmul_rn(x.z, a.c.z), __fmul_rn(y.z, a.s.z)),
                       __fadd_rn(__fmul_rn(x.w, a.c.w), __fmul_rn(y.w, a.s.w)));
}

__device__ __forceinline__ float4 bf16x4(uint2 u) {
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ uint2 raw_bf16x4(const __nv_bfloat16 *row, int lane) {
    return *reinterpret_cast<const uint2 *>(row + 4 * lane);
}
__device__ __forceinline__ float amax4(float m, float4 x) {
    return fmaxf(fmaxf(m, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
}

// rows cu[b] .. of sequence b, clamped into the packed tensors so that bad offsets stay memory-safe
__device__ __forceinline__ int2 new_rows(const AppendParams &p, int b) {
    const int r0 = min(max(p.cu[b], 0), p.total);
    return make_int2(r0, max(min(max(p.cu[b + 1], 0), p.total), r0));
}

// A (touched page, key head), both caches: the new tokens' largest value (rotated
// keys), the page's new scale, codes of its earlier tokens moved to that scale when
// it grew, then the new codes.  It is one CTA's own, or one warp's (kWarp: a few
// tokens per sequence, where a CTA's other warps would idle: 64 sequences of one
// token 14 against 4.5 us), so nothing is atomic; each warp's first HELD tokens stay in
// registers between the maximum and the codes, the rest are read again from L1/L2.
// CTAs past the page slots rotate q and tq: a warp takes one row of HEADS_PER_WARP
// heads, so that the row's angles, as many bytes as two heads' channels, are read
// once for them.  Bound by its bytes.
template <bool kWarp, int ROT>
__global__ void __launch_bounds__(APPEND_THREADS, 4) cache_append_kernel(const __grid_constant__ AppendParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_page_ctas = kWarp ? (p.n_slots * p.Hkv + APPEND_WARPS - 1) / APPEND_WARPS : p.n_slots * p.Hkv;
    if (ROT != ROT_NONE && (int)blockIdx.x >= n_page_ctas) {
        const int chunks = (p.total + APPEND_WARPS - 1) / APPEND_WARPS;
        const int u = (int)blockIdx.x - n_page_ctas, h0 = u / chunks * HEADS_PER_WARP;
        const int row = (u % chunks) * APPEND_WARPS + warp;
        if (row >= p.total) return;
        uint2 x[HEADS_PER_WARP], t[HEADS_PER_WARP];
#pragma unroll
        for (int i = 0; i < HEADS_PER_WARP; ++i) {
            const size_t off = ((size_t)min(h0 + i, p.H - 1) * p.total + row) * HD;
            x[i] = raw_bf16x4(p.q + off, lane);
            t[i] = p.tq ? raw_bf16x4(p.tq + off, lane) : make_uint2(0u, 0u);
        }
        int lo = 0, hi = p.n_seq;  // the last sequence that starts at or before the row: among 32 by a vote
        while (hi - lo > 32) {
            const int mid = (lo + hi) >> 1;
            if (p.cu[mid] <= row) lo = mid; else hi = mid;
        }
        const unsigned started = __ballot_sync(0xffffffffu, lo + lane < hi && p.cu[lo + lane] <= row);
        lo += started ? 31 - __clz(started) : 0;
        const int2 rows = new_rows(p, lo);
        if (row < rows.x || row >= rows.y) return;  // behind the last sequence: not written
        const Angles a = angles_of<ROT>(p, max(p.lens[lo], 0) + row - rows.x, lane);
#pragma unroll
        for (int i = 0; i < HEADS_PER_WARP; ++i) {
            if (h0 + i >= p.H) break;
            const size_t off = ((size_t)(h0 + i) * p.total + row) * HD + 4 * lane;
            const float4 y = rotate<ROT>(bf16x4(x[i]), a);
            *reinterpret_cast<uint2 *>(p.q_out + off) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
            if (p.tq) {
                const float4 z = rotate<ROT>(bf16x4(t[i]), a);
                *reinterpret_cast<uint2 *>(p.tq_out + off) = make_uint2(pack_bf16x2(z.x, z.y), pack_bf16x2(z.z, z.w));
            }
        }
        return;
    }
    // the slot'th touched page over all sequences, counted by every warp for itself
    const int unit = kWarp ? (int)blockIdx.x * APPEND_WARPS + warp : (int)blockIdx.x;
    const int slot = unit / p.Hkv, hk = unit - slot * p.Hkv;
    constexpr int STRIDE = kWarp ? 1 : APPEND_WARPS;  // tokens: every STRIDE'th from t0
    const int t0 = kWarp ? 0 : warp;
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
    if (b < 0) return;  // past the last touched page (the same for the whole unit)
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

    // this warp's tokens: kept + t0 + STRIDE i
    auto key = [&](int t) -> float4 {
        const float4 x = bf16x4(raw_bf16x4(krow + (size_t)(t - kept) * HD, lane));
        if constexpr (ROT == ROT_NONE)
            return x;
        else
            return rotate<ROT>(x, angles_of<ROT>(p, (int)(page0 + t), lane));
    };
    auto value = [&](int t) -> uint2 { return raw_bf16x4(vrow + (size_t)(t - kept) * HD, lane); };
    float ka = 0.f, va = 0.f;
    float4 kh[HELD];
    uint2 vh[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i) {  // (past the end: the last token once more, so that all loads are under way at once)
        const int t = min(kept + t0 + STRIDE * i, last - 1);
        kh[i] = key(t);
        vh[i] = value(t);
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        ka = amax4(ka, kh[i]);
        va = amax4(va, bf16x4(vh[i]));
    }
    for (int t = kept + t0 + STRIDE * HELD; t < last; t += STRIDE) {
        ka = amax4(ka, key(t));
        va = amax4(va, bf16x4(value(t)));
    }
    // positive floats order like their bits
    const uint32_t kb = __reduce_max_sync(0xffffffffu, __float_as_uint(ka));
    const uint32_t vb = __reduce_max_sync(0xffffffffu, __float_as_uint(va));
    const size_t sc = (size_t)id * p.Hkv + hk;
    // the old scales, read before any thread writes the new ones; a page that starts here has none
    const int ek_old = kept > 0 ? exponent_of(p.ks[sc]) : SCALE_MIN, ev_old = kept > 0 ? exponent_of(p.vs[sc]) : SCALE_MIN;
    uint32_t km = kb, vm = vb;
    if constexpr (kWarp) {
        __syncwarp();
    } else {
        __shared__ uint32_t s_k[APPEND_WARPS], s_v[APPEND_WARPS];
        if (lane == 0) {
            s_k[warp] = kb;
            s_v[warp] = vb;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < APPEND_WARPS; ++w) {
            km = max(km, s_k[w]);
            vm = max(vm, s_v[w]);
        }
    }
    const int ek = max(scale_exponent(__uint_as_float(km)), ek_old), ev = max(scale_exponent(__uint_as_float(vm)), ev_old);
    if (kWarp ? lane == 0 : threadIdx.x == 0) {
        p.ks[sc] = pow2(ek);
        p.vs[sc] = pow2(ev);
    }
    uint8_t *const kc = p.k8 + sc * p.page * HD, *const vc = p.v8 + sc * p.page * HD;
    auto moved = [&](uint8_t *codes, int from, int to) {
        const float r = from - to >= -126 ? pow2(from - to) : 0.f;
        for (int t = t0; t < kept; t += STRIDE) {
            uint32_t *const w = reinterpret_cast<uint32_t *>(codes + (size_t)t * HD) + lane;
            const float4 x = unpack_e4m3x4(*w);
            *w = pack_e4m3x4(make_float4(x.x * r, x.y * r, x.z * r, x.w * r));
        }
    };
    if (kept > 0 && ek > ek_old) moved(kc, ek_old, ek);
    if (kept > 0 && ev > ev_old) moved(vc, ev_old, ev);
    const float kr = pow2(-ek), vr = pow2(-ev);
    auto store = [&](int t, float4 x, float4 y) {
        reinterpret_cast<uint32_t *>(kc + (size_t)t * HD)[lane] =
            pack_e4m3x4(make_float4(x.x * kr, x.y * kr, x.z * kr, x.w * kr));
        reinterpret_cast<uint32_t *>(vc + (size_t)t * HD)[lane] =
            pack_e4m3x4(make_float4(y.x * vr, y.y * vr, y.z * vr, y.w * vr));
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int t = kept + t0 + STRIDE * i;
        if (t < last) store(t, kh[i], bf16x4(vh[i]));
    }
    for (int t = kept + t0 + STRIDE * HELD; t < last; t += STRIDE) store(t, key(t), bf16x4(value(t)));
}

// --------------------------------------------------------------- attention
// O, tO of n query tokens per sequence over the cache.  The cache carries no
// tangent, so with T = sum p dS V, tO = T / l - mu O.
//
// This is a decoding step: the work is to read the codes once, for a few query
// rows (the group's heads x n tokens).  Each warp takes runs of 32 tokens (two
// halves of 16, each inside one page), which the tensor-memory accelerator
// copies ahead into a ring of its own in shared memory, 128-byte swizzled.  The
// products have the 16 tokens, or 16 value channels, as rows and the query rows
// as their 8 columns,
//     S^T = K Q^T      [16 tokens][8]
//     O^T += V^T P^T   [128 channels][8]
// so that few query rows leave little of a product empty.  With a tangent the
// columns alternate q, tq: one thread holds S and dS of the same (row, key), and
// the columns of the second product alternate P, P dS, giving O and T at once.
// The codes become f16 operands in registers, two per instruction (m16n8k32 in
// e4m3 takes them as they are, but needs the queries in two parts and P in three,
// and measured slower: 174 instead of 132 us for 64 sequences of up to 8192
// tokens).  Bytes of two tokens' value rows pair up as A fragments, and P^T is
// turned by movmatrix.
// mma.sync rather than tcgen05 is a choice for few query rows, not a limit: in this
// orientation 128 tokens, or the 128 channels, would fill tcgen05's 128 rows, with 16
// and more query columns, but its operands would have to be converted into shared
// memory first.  That form is not built: chunks of many query tokens take every eight
// columns' products, and their conversions, anew.  Splits of a
// sequence are the CTAs of one cluster, which join their sums through distributed
// shared memory in one launch; or, for long contexts of few sequences, any number of
// CTAs that leave them in a workspace for a second kernel (make_plan in cache.cu says
// when).  Either way the order of additions is fixed.
//
// Operand ranges: queries and tangents are scaled by a power of two per row so
// that the largest lies in [1, 2) (bf16 channels are then exact but for those
// 2^-14 below it).  P is weighted by its page's value scale and a row's reference
// M covers both: it is set so that the largest weight is 2^7 and moves when one
// would pass 2^8.75, so weights 2^-21 below the row's largest start to lose bits.
// P dS is rounded with dS relative to r, a mean of dS over at least a sixteenth of
// the weight that the warp has summed so far, so that neither a nearly constant dS
// nor that of tokens that hardly count (far ones under a bias come first) costs
// bits; it has a power of two of its own, which rises with it and falls with the
// weights.  (An eighth in place of a sixteenth: 26.2 against 25.7 us for one sequence
// of 32760 tokens with 40 heads on 8; a unit that falls: 26.1; r of the first run
// alone: 24.9, but tO was lost where that run weighs little.)
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
    float cap_in, cap_w, cap_out; // of log2-unit scores y: tanh(z / c) = 1 - 2 / (1 + 2^(cap_in y)), z / c = cap_w y; c log2(e)
                                  // (0: no cap)
    float scale;
    int B, H, Hkv, group, n_pages, page, table_width, causal;
    int n;                        // query tokens per sequence (packed: of the longest)
    int tiles;                    // row tiles per (sequence, key head)
    int splits;                   // CTAs per unit
    float *partial;               // NULL: the CTAs of a unit are one cluster; else their sums, for cache_join_kernel
    CUtensorMap tm_k, tm_v;       // codes [rows][128], boxes of 16 rows
    unsigned long long bound_ns;
    unsigned page_magic;          // ceil(2^32 / (page / 16)): x / (page / 16) = umulhi(x, magic); 0 for pages of 16
};

// The least exponent of a value scale that the references follow (a page of zeros has 2^-100): 2^24 exponentials
// of at most 2^88.75 stay below 2^113, and their products with dS below 2^128 for dS up to 2^15 units.  Under
// smaller scales weights are at most 2^(8.75 + 80 - 100), which f16 holds to 2^-13 of the largest.
constexpr int EV_MIN = -80;
constexpr int EW_MIN = -120;                         // T's unit before any weight
constexpr int HALF_BYTES = 16 * HD;                  // 16 tokens of keys, or of values
constexpr int STAGE_BYTES = 4 * HALF_BYTES;          // 32 tokens: keys, then values
// statistics of a warp, or of the CTA: floats at ST_M + row etc.
constexpr int ST_M = 0, ST_L = 16, ST_G = 32, ST_R = 40, ST_E = 48, ST_UNIT = 56, ST_FLOATS = 64;
// shared memory of a CTA: the warps' rings of `stages` runs, a barrier per warp and
// stage and the CTA's abort flag, statistics of the warps and of the CTA
__host__ __device__ constexpr int bars_off(int warps, int stages) { return warps * stages * STAGE_BYTES; }
__host__ __device__ constexpr int stats_off(int warps, int stages) { return bars_off(warps, stages) + warps * stages * 8 + 16; }
__host__ __device__ constexpr int attn_smem(int warps, int stages) {
    return stats_off(warps, stages) + (warps + 1) * ST_FLOATS * 4;
}
static_assert(16 * HD * 4 <= STAGE_BYTES, "the sums of a warp fit a stage");
// a CTA's statistics and sums in a workspace: a unit has 8 nt columns
__host__ __device__ constexpr int part_floats(int nt) { return ST_FLOATS + 8 * nt * HD; }
constexpr int MOST_PARTS = 64;

// 2-D tiled load global -> shared, completion counted on `bar` (bytes)
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void *tmap, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same without an addend
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// four e4m3 codes as two f16x2; exact
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// an 8 x 8 matrix of 16-bit values, row lane / 4, columns 2 (lane % 4) + {0, 1}: its transpose
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// over the eight lanes of the same lane % 4
__device__ __forceinline__ float column_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float column_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ void axpy(float4 &y, float a, float4 x) {
    y.x = fmaf(a, x.x, y.x);
    y.y = fmaf(a, x.y, y.y);
    y.z = fmaf(a, x.z, y.z);
    y.w = fmaf(a, x.w, y.w);
}
// weight of sums at reference m against reference top
__device__ __forceinline__ float ref_weight(float m, float top) { return m == -INFINITY ? 0.f : ex2_approx(m - top); }
// e with |x| in [2^e, 2^(e + 1)), at most 119
__device__ __forceinline__ int binary_exponent(float x) {
    return min((int)((__float_as_uint(x) >> 23) & 255u) - 127, 119);
}
__device__ __forceinline__ float pow2_or_0(int e) { return e >= -126 ? pow2(e) : 0.f; }

// O, tO and lse of a row, channels 4 d4 .. 4 d4 + 3, from its sums: T is in units
// of 2^E, and like g relative to r and in units of the tangent row's scaling
template <bool kTan>
__device__ __forceinline__ void write_row(const AttnParams &p, size_t out, int d4, float4 so, float4 sT, float lt, float gt,
                                          float top, int E, float unit) {
    const float inv = lt > 0.f ? 1.f / lt : 0.f;  // a row that sees no key: zeros, lse = -infinity
    const float4 ov = make_float4(so.x * inv, so.y * inv, so.z * inv, so.w * inv);
    *reinterpret_cast<uint2 *>(p.o + out * HD + 4 * d4) = make_uint2(pack_bf16x2(ov.x, ov.y), pack_bf16x2(ov.z, ov.w));
    if constexpr (kTan) {
        const float mu = gt * inv, in = pow2(E) * inv;
        *reinterpret_cast<uint2 *>(p.to + out * HD + 4 * d4) =
            make_uint2(pack_bf16x2(unit * fmaf(-mu, ov.x, sT.x * in), unit * fmaf(-mu, ov.y, sT.y * in)),
                       pack_bf16x2(unit * fmaf(-mu, ov.z, sT.z * in), unit * fmaf(-mu, ov.w, sT.w * in)));
    }
    if (d4 == 0 && p.lse) p.lse[out] = lt > 0.f ? (top + __log2f(lt)) * 0.69314718055994531f : -INFINITY;
}

// NT column tiles of 8: with a tangent 4 NT query rows and their tangents, else 8 NT query rows.
// WARPS x STAGES: 4 x 2 (three CTAs per SM for one column tile, two for two), or
// 8 x 3 for launches of at most one CTA per SM, where a warp's own copies have to
// cover the latency.
template <bool kTan, int NT, int WARPS, int STAGES>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 4 ? (NT == 1 ? 3 : 2) : 1) cache_attn_kernel(const __grid_constant__ AttnParams p) {
    constexpr int ROWS = (kTan ? 4 : 8) * NT;  // query rows of a tile
    constexpr int R = kTan ? 1 : 2;            // query rows per thread and column tile
    constexpr int THREADS = 32 * WARPS, STATS_OFF = stats_off(WARPS, STAGES);
    constexpr int RING_BYTES = STAGES * STAGE_BYTES;  // per warp
    if (p.partial) asm volatile("griddepcontrol.launch_dependents;");  // the join's blocks wait for this grid's end
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (sbase & 1023u) {  // the swizzled copies need it (the same for every CTA)
        if (threadIdx.x == 0) atomicOr(&g_status_word, 2);
        return;
    }
    const int gr = lane >> 2, c = lane & 3;  // fragment row and column pair
    const int rank = (int)blockIdx.x % p.splits;
    const int unit = (int)blockIdx.x / p.splits;
    const int tile = unit % p.tiles, bh = unit / p.tiles;
    const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
    int n = p.n, first = 0;  // this sequence's query tokens and their first row
    int n_all = n;           // (packed: n of these are computed)
    if (p.cu) {
        first = min(max(p.cu[b], 0), p.total);
        n_all = max(min(max(p.cu[b + 1], 0), p.total) - first, 0);
        n = min(n_all, p.n);
    }
    const int n_rows = p.group * n;
    if (tile * ROWS >= n_rows) return;  // (the same for every CTA of the cluster)
    const int len = min(max(p.lens[b], 0), p.table_width * p.page);
    // this CTA's runs of 32 tokens
    const int runs = (len + 31) >> 5;
    const int per = (runs + p.splits - 1) / p.splits;
    const int run0 = min(rank * per, runs), run1 = min(run0 + per, runs);

    const uint32_t ring = sbase + (uint32_t)warp * RING_BYTES;
    const uint32_t bars = sbase + bars_off(WARPS, STAGES) + (uint32_t)warp * STAGES * 8u;
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(smem + bars_off(WARPS, STAGES) + WARPS * STAGES * 8);
    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < STAGES; ++s) mbar_init(bars + 8u * s, 2);  // lanes 0 and 1
        if (warp == 0) *abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    const int *const table = p.table + (size_t)b * p.table_width;
    const int halves = (len + 15) >> 4, per_page = p.page >> 4;
    auto page_index = [&](int half) -> int { return p.page_magic ? (int)__umulhi((unsigned)half, p.page_magic) : half; };
    // lane h < 2 looks after half h of every run: its page (-1: past the end, or no such page) ...
    auto page_of = [&](int run) -> int {
        if (lane >= 2 || run >= run1 || 2 * run + lane >= halves) return -1;
        const int id = table[page_index(2 * run + lane)];
        return (unsigned)id < (unsigned)p.n_pages ? id : -1;
    };
    // ... and its copy; returns its {key, value} scales (key -1, which no scale is: hidden)
    auto copy = [&](int run, int id, int stage) -> float2 {
        float2 sc = make_float2(-1.f, 0.f);
        if (lane < 2 && run < run1) {
            const uint32_t bar = bars + 8u * stage, d = ring + (uint32_t)(stage * STAGE_BYTES + lane * HALF_BYTES);
            if (id >= 0) {
                const int at = id * p.Hkv + hk, half = 2 * run + lane;
                const int y = at * p.page + (half - page_index(half) * per_page) * 16;
                mbar_arrive_expect_tx(bar, 2 * HALF_BYTES);
                tma_load_2d(d, &p.tm_k, bar, 0, y);
                tma_load_2d(d + 2 * HALF_BYTES, &p.tm_v, bar, 0, y);
                sc = make_float2(__ldg(p.ks + at), __ldg(p.vs + at));
            } else {
                mbar_arrive(bar);
            }
        }
        return sc;
    };
    float2 held[STAGES];  // scales of the runs in flight, the one being worked on first
    int id_next;          // page of the run after them
#pragma unroll
    for (int s = 0; s < STAGES; ++s) held[s] = copy(run0 + warp + s * WARPS, page_of(run0 + warp + s * WARPS), s);
    id_next = page_of(run0 + warp + STAGES * WARPS);

    // query fragments: column gr of each column tile; product w takes channels 32 c + 4 w
    // .. 32 c + 4 w + 3 of this lane
    uint32_t bq[NT][8][2];
    float unit_of[NT];  // power of two of the column's scaling, times the softmax scale
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = tile * ROWS + (kTan ? nt * 4 + (gr >> 1) : nt * 8 + gr);
        const bool live = r < n_rows;
        const int h = live ? hk * p.group + r / n : 0, t = live ? r % n : 0;
        const __nv_bfloat16 *src = (kTan && (gr & 1) ? p.tq : p.q) + (p.q_b * b + p.q_h * h + p.q_t * (first + t));
        uint4 raw[4];
        float amax = 0.f;
#pragma unroll
        for (int s = 0; s < 4; ++s)
            raw[s] = live ? *reinterpret_cast<const uint4 *>(src + 32 * c + 8 * s) : make_uint4(0u, 0u, 0u, 0u);
        float x[32];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const uint32_t u[4] = {raw[s].x, raw[s].y, raw[s].z, raw[s].w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                x[8 * s + 2 * w] = __uint_as_float(u[w] << 16);
                x[8 * s + 2 * w + 1] = __uint_as_float(u[w] & 0xffff0000u);
                amax = fmaxf(amax, fmaxf(fabsf(x[8 * s + 2 * w]), fabsf(x[8 * s + 2 * w + 1])));
            }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^e with amax in [2^e, 2^(e + 1))
        const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -120), 120);
        const float inv = pow2(-e);
        unit_of[nt] = pow2(e) * p.scale;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            bq[nt][w][0] = pack_f16x2(x[4 * w] * inv, x[4 * w + 1] * inv);
            bq[nt][w][1] = pack_f16x2(x[4 * w + 2] * inv, x[4 * w + 3] * inv);
        }
    }
    // this thread's rows: columns 2 c and 2 c + 1 (a row and its tangent, or two rows)
    float unit_q[NT][R], unit_t[NT], slope2[NT][R];
    int end[NT][R], pos[NT][R];  // keys 0 .. end - 1 are visible; the row's position
    int least = len;             // keys that every row of the warp sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float u0 = __shfl_sync(0xffffffffu, unit_of[nt], 8 * c), u1 = __shfl_sync(0xffffffffu, unit_of[nt], 8 * c + 4);
        unit_q[nt][0] = u0;
        if constexpr (!kTan) unit_q[nt][1] = u1;
        unit_t[nt] = u1;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = tile * ROWS + (kTan ? nt * 4 + c : nt * 8 + 2 * c + i);
            const bool live = r < n_rows;
            pos[nt][i] = len - n_all + (live ? r % n : 0);
            end[nt][i] = live && p.causal ? min(max(pos[nt][i] + 1, 0), len) : len;
            slope2[nt][i] = p.slopes && live ? p.slopes[hk * p.group + r / n] * 1.4426950408889634f : 0.f;
            least = min(least, end[nt][i]);
        }
    }
    least = __reduce_min_sync(0xffffffffu, least);

    float acc[NT][8][4];  // channels 16 gr + 2 j + {0, 1} (pairs of elements), columns 2 c + {0, 1}
    float m[NT][R], l[NT][R], g[NT], r0[NT], lr[NT];  // lr: the row's sum when r was set
    int ew[NT];    // T is in units of 2^ew
    float mw[NT];  // m when the unit was set
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nt][j][i] = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            m[nt][i] = -INFINITY;
            l[nt][i] = 0.f;
        }
        g[nt] = r0[nt] = lr[nt] = 0.f;
        ew[nt] = EW_MIN;
        mw[nt] = -INFINITY;
    }

    int stage = 0;
    uint32_t phase = 0;
    for (int run = run0 + warp; run < run1; run += WARPS) {
        if (!mbar_wait_warp(bars + 8u * stage, phase, abort_flag, p.bound_ns)) break;
        const uint32_t d = ring + (uint32_t)stage * STAGE_BYTES;
        float kscale[2], vscale[2];
        bool valid[2];  // (a half without a page is hidden)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            kscale[h] = __shfl_sync(0xffffffffu, held[0].x, h);
            vscale[h] = __shfl_sync(0xffffffffu, held[0].y, h);
            valid[h] = kscale[h] != -1.f;  // (a scale of 0 counts: its keys are zero)
        }

        // S^T of tokens gr (elements 0, 1) and gr + 8 (2, 3) of each half; two chains of four
        // products each
        float S[2][NT][4], S2[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // 16-byte units 2 c, 2 c + 1 of rows gr and gr + 8 (unit u of row r at u ^ (r & 7))
            const uint32_t dh = d + (uint32_t)(h * HALF_BYTES + gr * HD);
            const uint32_t u0 = (uint32_t)((2 * c) ^ gr) * 16u, u1 = (uint32_t)((2 * c + 1) ^ gr) * 16u;
            const uint4 x0 = ld_shared_u4(dh + u0), x1 = ld_shared_u4(dh + u1);
            const uint4 y0 = ld_shared_u4(dh + 8 * HD + u0), y1 = ld_shared_u4(dh + 8 * HD + u1);
            const uint32_t lo[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
            const uint32_t up[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
                e4m3x4_to_f16x2(lo[w], a0, a2);
                e4m3x4_to_f16x2(up[w], a1, a3);
                e4m3x4_to_f16x2(lo[4 + w], b0, b2);
                e4m3x4_to_f16x2(up[4 + w], b1, b3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (w == 0) {
                        mma_f16_first(S[h][nt], a0, a1, a2, a3, bq[nt][w][0], bq[nt][w][1]);
                        mma_f16_first(S2[h][nt], b0, b1, b2, b3, bq[nt][4 + w][0], bq[nt][4 + w][1]);
                    } else {
                        mma_f16(S[h][nt], a0, a1, a2, a3, bq[nt][w][0], bq[nt][w][1]);
                        mma_f16(S2[h][nt], b0, b1, b2, b3, bq[nt][4 + w][0], bq[nt][4 + w][1]);
                    }
                }
            }
        }
        // log2-unit scores y of this thread's rows at keys run * 32 + 16 h + gr + {0, 8}
        float y[2][NT][R][2], dS[2][NT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float klog = kscale[h] * 1.4426950408889634f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        y[h][nt][i][e] = (S[h][nt][2 * e + i] + S2[h][nt][2 * e + i]) * (klog * unit_q[nt][i]);
                    if constexpr (kTan) dS[h][nt][e] = (S[h][nt][2 * e + 1] + S2[h][nt][2 * e + 1]) * kscale[h];
                }
        }
        const bool partial = (run + 1) * 32 > least || !valid[0] || !valid[1];
        auto hide = [&](float as) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int i = 0; i < R; ++i)
                            if (!valid[h] || run * 32 + 16 * h + gr + 8 * e >= end[nt][i]) {
                                y[h][nt][i][e] = as;
                                if constexpr (kTan) dS[h][nt][e] = 0.f;  // (codes past the end may be NaN)
                            }
        };
        if (p.cap_out > 0.f) {
            // scores well below the cap by the polynomial: the exponential's tanh is exact to 2^-23 absolute, which
            // a wide cap multiplies.  Hidden scores, which may come from anything, have no say in the choice.
            if (partial) hide(0.f);
            float most = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        most = fmax3(most, fabsf(y[h][nt][i][0]), fabsf(y[h][nt][i][1]));
            auto cap = [&](auto small) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < R; ++i) {
                            const float2 x = make_float2(y[h][nt][i][0], y[h][nt][i][1]);
                            float2 t, df;
                            if constexpr (decltype(small)::value)
                                cap2_small(x, p.cap_w, t, df);
                            else
                                cap2(x, p.cap_in, t, df);
                            y[h][nt][i][0] = t.x * p.cap_out;
                            y[h][nt][i][1] = t.y * p.cap_out;
                            if constexpr (kTan) {
                                dS[h][nt][0] *= df.x;
                                dS[h][nt][1] *= df.y;
                            }
                        }
            };
            if (__all_sync(0xffffffffu, most * p.cap_w <= CAP_SMALL))
                cap(std::true_type{});
            else
                cap(std::false_type{});
        }
        if (p.slopes) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const float dist = (float)(pos[nt][i] - run * 32 - 16 * h - gr);
                        y[h][nt][i][0] = fmaf(-slope2[nt][i], fabsf(dist), y[h][nt][i][0]);
                        y[h][nt][i][1] = fmaf(-slope2[nt][i], fabsf(dist - 8.f), y[h][nt][i][1]);
                    }
        }
        if (partial) hide(-INFINITY);
        // running references: weights 2^(y + ev - m), the largest 2^7 when set, at most 2^8.75 = 430.  exp2(y - m)
        // is 2^-ev times a weight: below EV_MIN its sums, and those of its products with dS, could pass 2^128
        const float ev[2] = {(float)max(exponent_of(vscale[0]), EV_MIN), (float)max(exponent_of(vscale[1]), EV_MIN)};
        bool need = false;
        float top[NT][R];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < R; ++i) {
                top[nt][i] = fmaxf(fmaxf(y[0][nt][i][0], y[0][nt][i][1]) + ev[0], fmaxf(y[1][nt][i][0], y[1][nt][i][1]) + ev[1]);
                need |= top[nt][i] > m[nt][i] + 8.75f;
            }
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float alpha[R];
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float mx = column_max(top[nt][i]) - 7.f;
                    alpha[i] = 1.f;
                    if (mx > m[nt][i]) {
                        alpha[i] = ex2_approx(m[nt][i] - mx);
                        m[nt][i] = mx;
                    }
                    l[nt][i] *= alpha[i];
                    if constexpr (kTan) {
                        g[nt] *= alpha[i];
                        lr[nt] *= alpha[i];
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[nt][j][i] *= alpha[kTan ? 0 : (i & 1)];
            }
        }
        float pe[2][NT][R][2];  // exp2(y - m)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float ref = m[nt][i] == -INFINITY ? 0.f : m[nt][i];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) pe[h][nt][i][e] = ex2_approx(y[h][nt][i][e] - ref);
                l[nt][i] += (pe[0][nt][i][0] + pe[0][nt][i][1]) + (pe[1][nt][i][0] + pe[1][nt][i][1]);
            }
        if constexpr (kTan) {
            // r, a mean of dS over at least a sixteenth of the row's weight so far: by the time the sum has grown
            // sixteenfold, one of the row's eight threads holds more than twice the sum at r
            bool grown = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) grown |= l[nt][0] > 2.f * lr[nt];
            if (__any_sync(0xffffffffu, grown)) {
                float dr[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float s = g[nt];  // with this run's
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 2; ++e) s = fmaf(pe[h][nt][0][e], dS[h][nt][e] - r0[nt], s);
                    s = column_sum(s);
                    lr[nt] = column_sum(l[nt][0]);
                    const float r = lr[nt] > 0.f ? r0[nt] + s / lr[nt] : r0[nt];
                    dr[nt] = r - r0[nt];
                    r0[nt] = r;
                }
                if (run != run0 + warp) {  // the sums of earlier runs move to the new r
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float now = (pe[0][nt][0][0] + pe[0][nt][0][1]) + (pe[1][nt][0][0] + pe[1][nt][0][1]);
                        g[nt] = fmaf(-dr[nt], l[nt][0] - now, g[nt]);
                        // sum p (dS - r') V = sum p (dS - r) V - (r' - r) sum p V, whose last product stays inside
                        // fp32 in these units with sums of up to 2^42
                        // The unit falls as far as the weights that it was set by have since m rose (T with them, so
                        // that it stays in range; by more than 2^126 it is nothing).
                        const int by = (int)fminf(m[nt][0] - mw[nt], (float)(ew[nt] - EW_MIN));
                        const int e = max(ew[nt] - by, binary_exponent(dr[nt]) - 80);
                        const float f = ew[nt] - e > 126 ? 0.f : pow2_or_0(ew[nt] - e), d = -dr[nt] * pow2(-e);
                        ew[nt] = e;
                        mw[nt] = m[nt][0];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            acc[nt][j][1] = fmaf(d, acc[nt][j][0], acc[nt][j][1] * f);
                            acc[nt][j][3] = fmaf(d, acc[nt][j][2], acc[nt][j][3] * f);
                        }
                    }
                }
            }
        }
        float wt[2][NT][2][2];  // the columns of P^T: [half][][column 2 c + i][token gr + 8 e]
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    wt[h][nt][0][e] = pe[h][nt][0][e] * vscale[h];
                    if constexpr (kTan) {
                        const float dc = dS[h][nt][e] - r0[nt];
                        g[nt] = fmaf(pe[h][nt][0][e], dc, g[nt]);
                        wt[h][nt][1][e] = wt[h][nt][0][e] * dc;
                    } else {
                        wt[h][nt][1][e] = pe[h][nt][R - 1][e] * vscale[h];
                    }
                }
        if constexpr (kTan) {  // P dS in units of 2^ew, at most 448 of them
            float most[NT];
            bool over = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                most[nt] = fmaxf(fmaxf(fabsf(wt[0][nt][1][0]), fabsf(wt[0][nt][1][1])),
                                 fmaxf(fabsf(wt[1][nt][1][0]), fabsf(wt[1][nt][1][1])));
                over |= most[nt] > 448.f * pow2(ew[nt]);
            }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float mx = column_max(most[nt]);
                    const int e = binary_exponent(mx) - 7;  // mx in [2^7, 2^8) units
                    if (e > ew[nt]) {
                        const float r = pow2_or_0(ew[nt] - e);
                        ew[nt] = e;
                        mw[nt] = m[nt][0];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            acc[nt][j][1] *= r;
                            acc[nt][j][3] *= r;
                        }
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float to_units = pow2(-ew[nt]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) wt[h][nt][1][e] *= to_units;
            }
        }
        uint32_t bp[2][NT][2];  // P^T: tokens 2 c, 2 c + 1 and 2 c + 8, 2 c + 9 of column gr
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    bp[h][nt][e] = transpose_8x8(pack_f16x2(wt[h][nt][0][e], wt[h][nt][1][e]));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // values of tokens 2c, 2c + 1, 2c + 8, 2c + 9, channels 16 gr .. 16 gr + 15; tokens past
            // the end may hold anything (also NaN codes) and are zeroed
            const uint32_t dh = d + (uint32_t)((2 + h) * HALF_BYTES + 2 * c * HD);
            const uint32_t u0 = (uint32_t)(gr ^ (2 * c)) * 16u, u1 = HD + (uint32_t)(gr ^ (2 * c + 1)) * 16u;
            uint4 v0 = ld_shared_u4(dh + u0), v1 = ld_shared_u4(dh + u1);
            uint4 v2 = ld_shared_u4(dh + 8 * HD + u0), v3 = ld_shared_u4(dh + 8 * HD + u1);
            if (!valid[h] || run * 32 + 16 * h + 16 > len) {
                const int left = valid[h] ? len - run * 32 - 16 * h - 2 * c : 0;
                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                if (left <= 0) v0 = zero;
                if (left <= 1) v1 = zero;
                if (left <= 8) v2 = zero;
                if (left <= 9) v3 = zero;
            }
            const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
            const uint32_t w2[4] = {v2.x, v2.y, v2.z, v2.w}, w3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                // channels 4 w .. 4 w + 3 of two tokens, interleaved: [c0 t, c0 t', c1 t, c1 t'], [c2 .., c3 ..]
                uint32_t a[8];
                e4m3x4_to_f16x2(__byte_perm(w0[w], w1[w], 0x5140), a[0], a[1]);
                e4m3x4_to_f16x2(__byte_perm(w0[w], w1[w], 0x7362), a[2], a[3]);
                e4m3x4_to_f16x2(__byte_perm(w2[w], w3[w], 0x5140), a[4], a[5]);
                e4m3x4_to_f16x2(__byte_perm(w2[w], w3[w], 0x7362), a[6], a[7]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_f16(acc[nt][2 * w], a[0], a[1], a[4], a[5], bp[h][nt][0], bp[h][nt][1]);
                    mma_f16(acc[nt][2 * w + 1], a[2], a[3], a[6], a[7], bp[h][nt][0], bp[h][nt][1]);
                }
            }
        }
        // this stage is free again: the run STAGES further on
        __syncwarp();
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) held[s] = held[s + 1];
        held[STAGES - 1] = copy(run + STAGES * WARPS, id_next, stage);
        id_next = page_of(run + (STAGES + 1) * WARPS);
        if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
        }
    }
    if (*abort_flag) {  // a wait gave up: let the copies in flight land before their memory is used again
        if (lane == 0)
            for (int s = 0; s < STAGES; ++s) mbar_wait_drain(bars + 8u * s, s < stage ? phase ^ 1u : phase, p.bound_ns);
    }
    __syncwarp();

    // each warp's sums into its ring, [columns][128]; its statistics beside them
    float *const mine = reinterpret_cast<float *>(smem + warp * RING_BYTES);
    float *const stats = reinterpret_cast<float *>(smem + STATS_OFF) + warp * ST_FLOATS;
    // the CTA's, in shared memory or the workspace
    float *const part_of = p.partial ? p.partial + (size_t)blockIdx.x * part_floats(NT) : nullptr;
    float *const cst = part_of ? part_of : reinterpret_cast<float *>(smem + STATS_OFF) + WARPS * ST_FLOATS;
    float *const csum = part_of ? part_of + ST_FLOATS : reinterpret_cast<float *>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < R; ++i) l[nt][i] = column_sum(l[nt][i]);
        if constexpr (kTan) g[nt] = column_sum(g[nt]);
#pragma unroll
        for (int col = 0; col < 2; ++col)
#pragma unroll
            for (int j = 0; j < 8; j += 2)
                *reinterpret_cast<float4 *>(mine + (nt * 8 + 2 * c + col) * HD + 16 * gr + 2 * j) =
                    make_float4(acc[nt][j][col], acc[nt][j][2 + col], acc[nt][j + 1][col], acc[nt][j + 1][2 + col]);
        if (gr == 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int row = kTan ? nt * 4 + c : nt * 8 + 2 * c + i;
                stats[ST_M + row] = m[nt][i];
                stats[ST_L + row] = l[nt][i];
            }
            if constexpr (kTan) {
                stats[ST_G + nt * 4 + c] = g[nt];
                stats[ST_R + nt * 4 + c] = r0[nt];
                reinterpret_cast<int *>(stats)[ST_E + nt * 4 + c] = ew[nt];
                if (warp == 0) cst[ST_UNIT + nt * 4 + c] = unit_t[nt];
            }
        }
    }
    __syncthreads();
    // the CTA's sums, in warp order, into warp 0's ring (or the workspace); its statistics into cst.
    // T and g of different r: sum p (dS - R) V = sum p (dS - r) V + (r - R) sum p V
    const float *const st = reinterpret_cast<const float *>(smem + STATS_OFF);
    for (int x = threadIdx.x; x < ROWS * HD / 4; x += THREADS) {
        const int row = x / (HD / 4), d4 = x % (HD / 4);
        float top = -INFINITY, Rc = 0.f;
        int Ec = EW_MIN;  // the largest unit, and none that r - R would overflow in
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            if (st[ST_FLOATS * w + ST_M + row] > top) {
                top = st[ST_FLOATS * w + ST_M + row];
                if (kTan) Rc = st[ST_FLOATS * w + ST_R + row];
            }
        if constexpr (kTan)
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
                Ec = max(Ec, max(reinterpret_cast<const int *>(st + ST_FLOATS * w)[ST_E + row],
                                 binary_exponent(st[ST_FLOATS * w + ST_R + row] - Rc)));
        float4 so = make_float4(0.f, 0.f, 0.f, 0.f), sT = so;
        float lt = 0.f, gt = 0.f;
        const int oc = (kTan ? 2 * row : row) * HD + 4 * d4;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float *const sw = st + ST_FLOATS * w;
            const float *const vw = reinterpret_cast<const float *>(smem + w * RING_BYTES);
            const float f = ref_weight(sw[ST_M + row], top);
            const float4 v = *reinterpret_cast<const float4 *>(vw + oc);
            lt = fmaf(f, sw[ST_L + row], lt);
            axpy(so, f, v);
            if constexpr (kTan) {
                const float dr = sw[ST_R + row] - Rc;
                gt = fmaf(f, fmaf(dr, sw[ST_L + row], sw[ST_G + row]), gt);
                axpy(sT, f * pow2_or_0(reinterpret_cast<const int *>(sw)[ST_E + row] - Ec),
                     *reinterpret_cast<const float4 *>(vw + oc + HD));
                axpy(sT, f * (dr * pow2(-Ec)), v);
            }
        }
        // (each place of warp 0's ring is read and written by this thread alone)
        *reinterpret_cast<float4 *>(csum + oc) = so;
        if constexpr (kTan) *reinterpret_cast<float4 *>(csum + oc + HD) = sT;
        if (d4 == 0) {
            cst[ST_M + row] = top;
            cst[ST_L + row] = lt;
            if constexpr (kTan) {
                cst[ST_G + row] = gt;
                cst[ST_R + row] = Rc;
                reinterpret_cast<int *>(cst)[ST_E + row] = Ec;
            }
        }
    }
    if (part_of) return;  // cache_join_kernel goes on
    auto cluster_sync = [&]() {
        if (p.splits > 1)
            asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        else
            __syncthreads();
    };
    cluster_sync();
    // The cluster's sums: the ranks share out the tile's rows x channels.  Each fetches all
    // ranks' statistics and its part of their sums by independent loads, into memory that the
    // rings no longer need, and adds them up in rank order.
    constexpr int KINDS = kTan ? 2 : 1;                  // O, T
    const int part = ROWS * (HD / 4) / p.splits;         // float4 places of a rank (splits divide 16)
    float *const ast = reinterpret_cast<float *>(smem + RING_BYTES);
    float4 *const sums = reinterpret_cast<float4 *>(smem + RING_BYTES + 16 * ST_FLOATS * 4);  // [rank][kind][part]
    for (int i = threadIdx.x; i < p.splits * ST_FLOATS; i += THREADS)
        ast[i] = ld_cluster(cluster_map(sbase + STATS_OFF + (WARPS * ST_FLOATS + (i & (ST_FLOATS - 1))) * 4u,
                                        (uint32_t)(i / ST_FLOATS)));
#pragma unroll 4
    for (int i = threadIdx.x; i < p.splits * KINDS * part; i += THREADS) {
        const int s = i / (KINDS * part), k = i / part % KINDS, x = rank * part + i % part;
        const int row = x / (HD / 4), d4 = x % (HD / 4);
        sums[i] = ld_cluster4(cluster_map(sbase, (uint32_t)s) + (uint32_t)((KINDS * row + k) * HD + 4 * d4) * 4u);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < part; i += THREADS) {
        const int x = rank * part + i, row = x / (HD / 4), d4 = x % (HD / 4), r = tile * ROWS + row;
        if (r >= n_rows) continue;
        float top = -INFINITY, Rt = 0.f;
        int Et = EW_MIN;
        for (int s = 0; s < p.splits; ++s) {
            const float *const a = ast + s * ST_FLOATS;
            if (a[ST_M + row] > top) {
                top = a[ST_M + row];
                if (kTan) Rt = a[ST_R + row];
            }
        }
        if constexpr (kTan)
            for (int s = 0; s < p.splits; ++s)
                Et = max(Et, max(__float_as_int(ast[s * ST_FLOATS + ST_E + row]),
                                 binary_exponent(ast[s * ST_FLOATS + ST_R + row] - Rt)));
        float4 so = make_float4(0.f, 0.f, 0.f, 0.f), sT = so;
        float lt = 0.f, gt = 0.f;
        for (int s = 0; s < p.splits; ++s) {
            const float *const a = ast + s * ST_FLOATS;
            const float f = ref_weight(a[ST_M + row], top);
            const float4 o4 = sums[s * KINDS * part + i];
            lt = fmaf(f, a[ST_L + row], lt);
            axpy(so, f, o4);
            if constexpr (kTan) {
                const float dr = a[ST_R + row] - Rt;
                gt = fmaf(f, fmaf(dr, a[ST_L + row], a[ST_G + row]), gt);
                axpy(sT, f * pow2_or_0(__float_as_int(a[ST_E + row]) - Et), sums[(s * KINDS + 1) * part + i]);
                axpy(sT, f * (dr * pow2(-Et)), o4);
            }
        }
        const int h = hk * p.group + r / n, t = r % n;
        write_row<kTan>(p, (size_t)(p.o_b * b + p.o_h * h + first + t), d4, so, sT, lt, gt, top, Et,
                        kTan ? cst[ST_UNIT + row] : 0.f);
    }
    cluster_sync();  // no CTA leaves while another still reads its sums
}

// Joins the parts that the CTAs of a unit left in the workspace: a block per
// query row, a lane per four channels, a warp per eighth of the parts; added up
// in a fixed order.  Launched beside the attention kernel, whose end it waits for.
constexpr int JOIN_WARPS = 8;
template <bool kTan, int NT>
__global__ void __launch_bounds__(32 * JOIN_WARPS) cache_join_kernel(const __grid_constant__ AttnParams p) {
    constexpr int ROWS = (kTan ? 4 : 8) * NT, PART = part_floats(NT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = (int)blockIdx.x % ROWS, unit = (int)blockIdx.x / ROWS;
    const int tile = unit % p.tiles, bh = unit / p.tiles;
    const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
    int n = p.n, first = 0;
    if (p.cu) {
        first = min(max(p.cu[b], 0), p.total);
        n = min(max(min(max(p.cu[b + 1], 0), p.total) - first, 0), p.n);
    }
    const int r = tile * ROWS + row;
    if (r >= p.group * n) return;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float *const parts = p.partial + (size_t)unit * p.splits * PART;
    float top = -INFINITY, Rt = 0.f;
    float ms[MOST_PARTS / 32], rs[MOST_PARTS / 32];
    int es[MOST_PARTS / 32], Et = EW_MIN;
#pragma unroll
    for (int i = 0; i < MOST_PARTS / 32; ++i) {
        const int s = 32 * i + lane;
        const float *const a = parts + (size_t)s * PART;
        ms[i] = s < p.splits ? a[ST_M + row] : -INFINITY;
        rs[i] = kTan && s < p.splits ? a[ST_R + row] : 0.f;
        es[i] = kTan && s < p.splits ? __float_as_int(a[ST_E + row]) : EW_MIN;
    }
#pragma unroll
    for (int i = 0; i < MOST_PARTS / 32; ++i) {  // the largest reference, and r of the first part that has it
        float m = ms[i];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        if (m > top) {
            top = m;
            Rt = __shfl_sync(0xffffffffu, rs[i], __ffs(__ballot_sync(0xffffffffu, ms[i] == m)) - 1);
        }
    }
    if constexpr (kTan) {
#pragma unroll
        for (int i = 0; i < MOST_PARTS / 32; ++i)
            Et = max(Et, __reduce_max_sync(0xffffffffu, 32 * i + lane < p.splits
                                                            ? max(es[i], binary_exponent(rs[i] - Rt)) : EW_MIN));
    }
    float4 so = make_float4(0.f, 0.f, 0.f, 0.f), sT = so;
    float lt = 0.f, gt = 0.f;
#pragma unroll 4
    for (int s = warp; s < p.splits; s += JOIN_WARPS) {
        const float *const a = parts + (size_t)s * PART;
        const float *const v = a + ST_FLOATS + (kTan ? 2 * row : row) * HD + 4 * lane;
        const float4 o4 = *reinterpret_cast<const float4 *>(v);
        const float f = ref_weight(a[ST_M + row], top);
        lt = fmaf(f, a[ST_L + row], lt);
        axpy(so, f, o4);
        if constexpr (kTan) {
            const float4 t4 = *reinterpret_cast<const float4 *>(v + HD);
            const float dr = a[ST_R + row] - Rt;
            gt = fmaf(f, fmaf(dr, a[ST_L + row], a[ST_G + row]), gt);
            axpy(sT, f * pow2_or_0(__float_as_int(a[ST_E + row]) - Et), t4);
            axpy(sT, f * (dr * pow2(-Et)), o4);
        }
    }
    __shared__ float4 s_o[JOIN_WARPS][32], s_t[JOIN_WARPS][32];
    __shared__ float s_l[JOIN_WARPS], s_g[JOIN_WARPS];
    s_o[warp][lane] = so;
    if constexpr (kTan) s_t[warp][lane] = sT;
    if (lane == 0) {
        s_l[warp] = lt;
        s_g[warp] = gt;
    }
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < JOIN_WARPS; ++w) {
        axpy(so, 1.f, s_o[w][lane]);
        if constexpr (kTan) axpy(sT, 1.f, s_t[w][lane]);
        lt += s_l[w];
        gt += s_g[w];
    }
    const int h = hk * p.group + r / n, t = r % n;
    write_row<kTan>(p, (size_t)(p.o_b * b + p.o_h * h + first + t), lane, so, sT, lt, gt, top, Et,
                    kTan ? parts[ST_UNIT + row] : 0.f);
}

}  // namespace cache
}  // namespace ajvp
