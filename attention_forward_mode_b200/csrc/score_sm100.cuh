// score_sm100.cuh -- score modifications shared by the forward and backward
// tensor-core kernels: a tanh cap, a bias by distance, an interval of visible
// keys per query row, and key heads shared by groups of query heads.
//
// With z = s Q K^T and dz = s (tQ K^T + Q tK^T) the modified scores are
//     S_ij = c tanh(z_ij / c) - slope_h |i + Lk - Lq - j|,   dS_ij = (1 - tanh^2(z_ij / c)) dz_ij
// and query row i of sequence b sees the keys begin[b][i] <= j < end[b][i].
// An interval per row is enough for prefix, document, frame-causal, causal
// and sliding-window masks, costs two integers per row whatever the mask, and
// gives every tile the range of the other side's tiles that it has to visit.
#pragma once

#include <climits>

#include "ptx_sm100.cuh"

namespace ajvp {

// MASK bits of the scored kernels (beside those of the kernels' own)
constexpr int MASK_SCORED = 8, MASK_CAP = 16, MASK_BIAS = 32;
// Forward, capped scores whose log2-unit cap is at most FIXED_CAP: |c log2(e) tanh| <= FIXED_CAP
// bounds every score before its bias, so each row keeps one reference for all
// its keys (the largest bias among them) in place of a running maximum: weights
// lie within 2^-80 .. 2^80 of it before the bias, inside the range of fp32 and
// bf16 with room for sums of 2^24 keys.  No maxima, no exchange of them between
// the softmax groups, no rescaling.
constexpr int MASK_FIXED = 64;
constexpr float FIXED_CAP = 80.f;

struct Score {
    const int *begin, *end;  // [B][Lq] visible keys of each query row, or NULL: 0 / Lk
    const float *slopes;     // [H] distance slopes (MASK_BIAS)
    const int2 *qrange;      // backward: [B][n_rtiles] first and end query row that sees a key of the 128-key tile
                             // (NULL: every row)
    float cap_in;            // 2 s log2(e) / c: tanh(z / c) = 1 - 2 / (1 + 2^(cap_in x)) of a raw score x = z / s
    float cap_w;             // s / c: z / c = cap_w x
    float cap_out;           // c log2(e): the capped score in log2 units is cap_out tanh
    float cap_second;        // 2 / c
    int H, Hkv, group;       // query heads, key heads, query heads per key head
    int slabs;               // (batch, head) slabs whose row tiles are scheduled together
};

// the visible keys of one query row, inside [0, Lk]; rows past the end see none
__device__ __forceinline__ int2 row_bounds(const Score &sc, int b, int row, int Lq, int Lk) {
    if (row >= Lq) return make_int2(0, 0);
    const size_t i = (size_t)b * (size_t)Lq + (size_t)row;
    const int lo = sc.begin ? max(sc.begin[i], 0) : 0;
    const int hi = sc.end ? min(sc.end[i], Lk) : Lk;
    return make_int2(lo, hi);
}

// The smallest interval that holds the visible keys of rows row0 .. row0 + 127
// (0, 0 if none sees any); every thread of the CTA calls it.  scratch: eight
// ints of shared memory.
__device__ __forceinline__ int2 tile_key_range(const Score &sc, int b, int row0, int Lq, int Lk, int *scratch) {
    if (!sc.begin && !sc.end) return make_int2(0, Lk);
    int *const s_lo = scratch, *const s_hi = scratch + 4;
    const int warp = threadIdx.x >> 5;
    if (warp < 4) {
        const int2 r = row_bounds(sc, b, row0 + (int)threadIdx.x, Lq, Lk);
        const bool any = r.x < r.y;
        const int lo = __reduce_min_sync(0xffffffffu, any ? r.x : INT_MAX);
        const int hi = __reduce_max_sync(0xffffffffu, any ? r.y : 0);
        if ((threadIdx.x & 31) == 0) {
            s_lo[warp] = lo;
            s_hi[warp] = hi;
        }
    }
    __syncthreads();
    const int lo = min(min(s_lo[0], s_lo[1]), min(s_lo[2], s_lo[3]));
    const int hi = max(max(s_hi[0], s_hi[1]), max(s_hi[2], s_hi[3]));
    return hi > 0 ? make_int2(lo, hi) : make_int2(0, 0);
}

// Forward, biased scores without a cap: the running reference takes the largest
// raw score of a tile's 64 keys and, separately, their largest bias.  Their sum
// is above every score of the tile by at most 63 |slope| log2(e) more than it
// need be, so up to this many log2 units the row's largest weight stays a normal
// number 2^24 times above the smallest; steeper slopes form each score before the
// maximum (one more packed operation and a dependence per score ahead of the
// exchange of the maxima).
constexpr float STEEP_LOG2 = 100.f;

// the largest bias -slope2 |pos - j| over the keys lo <= j < hi (0 without keys)
__device__ __forceinline__ float largest_bias(float slope2, int pos, int lo, int hi) {
    if (lo >= hi) return 0.f;
    const float near = (float)max(max(lo - pos, pos - (hi - 1)), 0);
    const float far = (float)max(abs(pos - lo), abs(pos - (hi - 1)));
    return fmaxf(-slope2 * near, -slope2 * far);
}

// bits i of a 32-wide tile with lo <= i < hi
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
    const uint32_t below_hi = hi <= 0 ? 0u : (hi >= 32 ? 0xffffffffu : (1u << hi) - 1u);
    const uint32_t below_lo = lo <= 0 ? 0u : (lo >= 32 ? 0xffffffffu : (1u << lo) - 1u);
    return below_hi & ~below_lo;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// tanh(z / c) of two raw scores, and 1 - tanh^2.  With e = exp(2 z / c) and
// r = 1 / (1 + e): tanh = 1 - 2 r and 1 - tanh^2 = 4 r (1 - r).  The error is
// a few 2^-24 absolute (the scores need absolute accuracy: c tanh enters an
// exponential), e = infinity gives r = 0.
__device__ __forceinline__ void cap2(float2 x, float cap_in, float2 &t, float2 &df) {
    const float2 y = __fmul2_rn(x, make_float2(cap_in, cap_in));
    const float2 r = make_float2(rcp_approx(1.f + ex2_approx(y.x)), rcp_approx(1.f + ex2_approx(y.y)));
    t = __ffma2_rn(r, make_float2(-2.f, -2.f), make_float2(1.f, 1.f));
    const float2 r4 = __fmul2_rn(r, make_float2(4.f, 4.f));
    df = __ffma2_rn(r4, make_float2(-r.x, -r.y), r4);
}

// The same where |z / c| <= CAP_SMALL, without the special-function unit (two
// of whose operations per score are what bounds the elementwise warps): with
// w = z / c, tanh w = w P(w^2), P the polynomial of degree 4 that minimises the
// largest error on [-CAP_SMALL, CAP_SMALL] (fitted by the Remez exchange, 3e-8
// absolute).  A warp takes it when every score that it holds is that small;
// scores under a cap that shapes only their tail are.
constexpr float CAP_SMALL = 0.625f;
__device__ __forceinline__ void cap2_small(float2 x, float cap_w, float2 &t, float2 &df) {
    const float2 w = __fmul2_rn(x, make_float2(cap_w, cap_w));
    const float2 v = __fmul2_rn(w, w);
    float2 r = __ffma2_rn(v, make_float2(0.014530068f, 0.014530068f), make_float2(-0.051362868f, -0.051362868f));
    r = __ffma2_rn(r, v, make_float2(0.13291031f, 0.13291031f));
    r = __ffma2_rn(r, v, make_float2(-0.33330483f, -0.33330483f));
    r = __ffma2_rn(r, v, make_float2(0.99999946f, 0.99999946f));
    t = __fmul2_rn(r, w);
    df = __ffma2_rn(t, make_float2(-t.x, -t.y), make_float2(1.f, 1.f));
}
template <bool kSmall>
__device__ __forceinline__ void cap2(const Score &sc, float2 x, float2 &t, float2 &df) {
    if constexpr (kSmall)
        cap2_small(x, sc.cap_w, t, df);
    else
        cap2(x, sc.cap_in, t, df);
}

// every score that the warp holds is inside the polynomial's range (a NaN stays one in either form)
template <int N>
__device__ __forceinline__ bool cap_all_small(const Score &sc, const uint32_t (&x)[N]) {
    float m[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        m[0] = fmax3(m[0], fabsf(__uint_as_float(x[i])), fabsf(__uint_as_float(x[i + 1])));
        m[1] = fmax3(m[1], fabsf(__uint_as_float(x[i + 2])), fabsf(__uint_as_float(x[i + 3])));
    }
    return __all_sync(0xffffffffu, fmaxf(m[0], m[1]) * fabsf(sc.cap_w) <= CAP_SMALL);
}

// [B][n_ktiles] query rows (first, end) that see a key of each 128-key tile,
// for the key-side kernels; a block of 256 threads calls it per sequence and tile (`index`).
__device__ __forceinline__ void query_range(const Score &sc, int Lq, int Lk, int2 *out, int index) {
    const int n_ktiles = (Lk + 127) / 128, b = index / n_ktiles;
    const int k0 = (index - b * n_ktiles) * 128;
    const int k1 = min(k0 + 128, Lk);
    int first = INT_MAX, end = 0;
    for (int q = (int)threadIdx.x; q < Lq; q += 256 * 8) {  // eight rows' loads under way at once
        int2 r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = row_bounds(sc, b, q + 256 * i, Lq, Lk);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (max(r[i].x, k0) < min(r[i].y, k1)) {
                first = min(first, q + 256 * i);
                end = q + 256 * i + 1;
            }
    }
    __shared__ int s_first[8], s_end[8];
    first = __reduce_min_sync(0xffffffffu, first);
    end = __reduce_max_sync(0xffffffffu, end);
    if ((threadIdx.x & 31) == 0) {
        s_first[threadIdx.x >> 5] = first;
        s_end[threadIdx.x >> 5] = end;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) {
            first = min(first, s_first[w]);
            end = max(end, s_end[w]);
        }
        out[index] = end > 0 ? make_int2(first, end) : make_int2(0, 0);
    }
}

}  // namespace ajvp
