// Matrix product over a quantised weight, with bias, activation and residual in its epilogue:
//   y[m, n] = act(sum_k x[m, k] w[n, k] + b[n]) + r[m, n]
// for a weight as the checkpoint stores it (FP8_TENSOR, FP8_BLOCK128, NVFP4, MXFP8, MXFP4) and rows x in
// bf16 or fp16, or in e4m3 with scales (FP8_ROW, FP8_GROUP128, MXFP8).
//
// Arithmetic.  w[n, k] is the code's value times its scales, not rounded to bf16 as a decoded weight is.
// Every product is exact and every sum is kept in fp32, but for the f8f6f4 instructions below:
//  * dense x: e4m3 and e2m1 codes, an e2m1 code times its e4m3 block scale (at most 6 significant
//    bits) and a code times a power of two are exact in bf16; the first three are exact in fp16 too, so the
//    weight enters the bf16 or fp16 matrix instructions without rounding.  fp16 rows against an MX
//    weight, whose scales reach beyond fp16, are split into two bf16 terms (x = hi + lo, exact).  An MX value outside bf16's range
//    is the exception: 2^128 or more (e4m3 under scales from 2^120 on, e2m1 under 2^126 and 2^127) becomes an infinity, and what
//    lies below 2^-126 a multiple of 2^-133 (e4m3 under 2^-125 and less; e2m1 loses nothing).
//  * e4m3 x: widened to bf16 (times its E8M0 scale) like the weight; or, for bf16 outputs of more than 64 rows,
//    the f8f6f4 matrix instructions, which run at twice the rate and apply the E8M0 scales of both sides
//    themselves.  Of 16 products that lie in one lane these cut what is below 2^-13 of the largest (measured: such
//    a product next to a larger one is lost; across lanes the sum is whole): at most 15 * 2^-13 of that largest product
//    per 16.  Measured under a residual that takes the result away, relative to the results' root mean square: 2e-5 on average and
//    4e-4 at worst for normally distributed weights and rows (K 1056 to 25600; e2m1 weights 7e-6 and 3e-4), 6e-5 and 3e-3 where
//    the codes spread evenly over all binades.  A bf16 result's own rounding is 1.1e-3 of itself on average and 2^-9 at most; an
//    fp16 result's, 1.4e-4, is not far enough above, so fp16 outputs, like fp32 ones, keep fp32 sums (2e-7 on average).
//  * fp32 scales (per tensor, per row, per 128 x 128 block, NVFP4's global one) multiply fp32 sums.
// The result is rounded once, to the output type.
//
// The weight is the A operand of the matrix instructions (its rows are the D rows), so a lane holds four
// consecutive output columns of one row of y and stores them together.
//
// Four kernels:
//  * linear_one: m = 1, dot products on the vector unit at the rate the weight arrives.
//  * linear_few: m <= 16.  Each wavefront streams its part of K for one or two 16-row groups of the weight straight
//    into registers and the matrix instructions, the wavefronts of a workgroup join in LDS.
//  * linear_tile: tiles of y, x and the weight staged through LDS as stored, one barrier per step of K and up to three steps on
//    their way; the weight is decoded on its way from LDS to the matrix instructions.
//  * linear_join: adds the fp32 partial results where K was split over workgroups, in a fixed order.
#pragma once

#include <type_traits>

#include "linear.h"
#include "matrix_codes.h"

namespace st_linear_impl {
namespace {

using namespace st_dev;

// ------------------------------------------------------------------------- epilogue

// Columns n..n+3 of row m from their sums (the kind's tensor-wide scales not yet applied).
template <int X, int WK>
__device__ __forceinline__ void finish(const Args& a, uint32_t m, uint32_t n, f32x4 v) {
    if (m >= a.m || n >= a.n) return;
    float s = 1.0f;
    if constexpr (WK == ST_KIND_FP8_TENSOR) s = *reinterpret_cast<const float*>(a.ws);
    if constexpr (WK == ST_KIND_NVFP4) s = *reinterpret_cast<const float*>(a.ws2);
    const uint32_t cnt = a.n - n < 4 ? a.n - n : 4;
    float y[4];
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
        y[i] = v[i];
        if constexpr (WK == ST_KIND_FP8_TENSOR || WK == ST_KIND_NVFP4) y[i] *= s;
        if constexpr (X == ST_X_FP8_ROW) y[i] *= reinterpret_cast<const float*>(a.xs)[m];
    }
    if (a.bias) {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            if (i < cnt) y[i] += load_as_f32(a.bias, a.bias_type, n + i);
    }
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) y[i] = activate(y[i], a.act);
    const uint64_t o = uint64_t(m) * a.out_pitch + n;
    if (a.res) {
        const uint64_t r = uint64_t(m) * a.res_pitch + n;
        if (a.vec && cnt == 4) {
            float t[4];
            load4_as_f32(a.res, a.res_type, r, t);
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) y[i] += t[i];
        } else {
            for (uint32_t i = 0; i < cnt; ++i) y[i] += load_as_f32(a.res, a.res_type, r + i);
        }
    }
    if (a.vec && cnt == 4) store4(a.out, a.out_type, o, y);
    else
        for (uint32_t i = 0; i < cnt; ++i) store_as(a.out, a.out_type, o + i, y[i]);
}

// A workgroup's result for columns n..n+3 of row m: the output, or this split's partial sums.
template <int X, int WK>
__device__ __forceinline__ void emit(const Args& a, uint32_t split, uint32_t m, uint32_t n, f32x4 v) {
    if (!a.part) return finish<X, WK>(a, m, n, v);
    if (m >= a.m || n >= a.n) return;
    float* p = a.part + (uint64_t(split) * a.m + m) * a.n + n;
    if ((a.n & 3) == 0) *reinterpret_cast<f32x4*>(p) = v;
    else
        for (uint32_t i = 0; i < 4 && n + i < a.n; ++i) p[i] = v[i];
}

template <int X, int WK>
__global__ __launch_bounds__(256) void linear_join(Args a) {
    const uint32_t q = (a.n + 3) / 4;
    const uint64_t i = uint64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= uint64_t(q) * a.m) return;
    const uint32_t m = uint32_t(i / q), n = uint32_t(i % q) * 4;
    f32x4 v = {0, 0, 0, 0};
    for (uint32_t s = 0; s < a.splits; ++s) {
        const float* p = a.part + (uint64_t(s) * a.m + m) * a.n + n;
        if ((a.n & 3) == 0) v += *reinterpret_cast<const f32x4*>(p);
        else
            for (uint32_t j = 0; j < 4 && n + j < a.n; ++j) v[j] += p[j];
    }
    finish<X, WK>(a, m, n, v);
}

// How dense x meets the weight: fp16 operands, or bf16 with fp16 x split in two terms.
template <int X, int WK>
struct Dense {
    static constexpr bool F16 = X == ST_X_F16 && !is_mx(WK), SPLIT = X == ST_X_F16 && is_mx(WK);
};

// ------------------------------------------------------------------------- one row

// m = 1: dot products on the vector unit.  Bound by the weight's bytes (NVFP4 [5120, 25600], 73.8 MB: 15.4-16.2 us, 4.6-4.8 TB/s;
// reading as many bytes and nothing else takes 13.9).  A wavefront takes a slice of K, 16 bytes of a weight row per lane, for R
// weight rows: its loads are contiguous, all R of them are in flight together, and its part of x stays in
// registers.  Decoding costs half an instruction per weight and multiplying another half (two-element dot
// products into fp32); a block's scale multiplies the block's sum.  (16x16x32 matrix instructions leave 15 of 16 columns empty for one
// token, want NVFP4 weights multiplied by their scales first, 2 instructions each, and x once per 16 weight rows.)
// The lanes' sums fold together within the wavefront, the slices' sums in LDS.
template <int X_, int WK_>
struct One {
    static constexpr int X = X_, WK = WK_, R = kOneRows;     // weight rows per wavefront
    static constexpr bool Q = is_q(X), FP4 = is_fp4(WK), GROUPED = WK == ST_KIND_FP8_BLOCK128;
    static constexpr int E = FP4 ? 32 : 16;          // elements of K per lane
    static constexpr int SLICE = 64 * E;
    static constexpr int PAIRS = E / 2;
};

template <bool F16>
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
    if constexpr (F16) return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, a), __builtin_bit_cast(f16x2, b), c, false);
    else return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c, false);
}

// Sum over the 64 lanes of each of N values: v[0] of lane l becomes the total of value l % N.  Each step halves the values a lane
// holds by handing the other half to the lane across.
template <int N>
__device__ __forceinline__ float fold(float* v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int half = N / 2; half >= 1; half /= 2) {
        const bool up = (lane & half) != 0;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float keep = up ? v[i + half] : v[i], give = up ? v[i] : v[i + half];
            v[i] = keep + __shfl_xor(give, half);
        }
    }
#pragma unroll
    for (int o = N; o < 64; o *= 2) v[0] += __shfl_xor(v[0], o);
    return v[0];
}

constexpr int kOneWaves = 4;

template <class F>
__global__ __launch_bounds__(64 * kOneWaves) void linear_one(Args a) {
    constexpr int X = F::X, WK = F::WK, R = F::R, E = F::E, PAIRS = F::PAIRS;
    using D = Dense<X, WK>;
    __shared__ __align__(16) float joined[kOneWaves][R];
    const int lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const uint32_t n0 = blockIdx.x * R;
    const uint32_t w_row = F::FP4 ? a.k / 2 : a.k, ws_row = a.k / (WK == ST_KIND_NVFP4 ? 16 : 32);
    const uint32_t groups = (a.k + 127) / 128;
    float acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = 0.0f;

    for (uint32_t k0 = wave * F::SLICE; k0 < a.k; k0 += waves * F::SLICE) {
        const uint32_t k = k0 + lane * E;
        const bool in = k < a.k;          // lanes behind K's end hold zeros,
        const bool all = k + E <= a.k;    // and the lane that it cuts the rest of its row
        u32x4 w[R];
        uint32_t ws[R];
        // rows past the last are read as the last one; nothing of them is stored
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t n = n0 + r < a.n ? n0 + r : a.n - 1;
            const uint8_t* pw = a.w + uint64_t(n) * w_row;
            const uint8_t* ps = a.ws + uint64_t(n) * ws_row;
            const uint32_t at = F::FP4 ? k / 2 : k;
            w[r] = u32x4{0, 0, 0, 0};
            ws[r] = 0;
            if (all) w[r] = *reinterpret_cast<const u32x4_any*>(pw + at);
            if constexpr (WK == ST_KIND_NVFP4) {
                if (all) ws[r] = *reinterpret_cast<const u16_any*>(ps + k / 16);
            } else if constexpr (is_mx(WK)) {
                if (in) ws[r] = ps[k / 32];
            }
            if constexpr (!is_mx(WK)) {
                if (in && !all) {
                    w[r] = load_chunk(pw + at, int64_t(w_row) - at);
                    if constexpr (WK == ST_KIND_NVFP4) ws[r] = ps[k / 16];
                }
            }
        }
        uint32_t x[PAIRS], xl[D::SPLIT ? PAIRS : 1];
        const uint8_t* px = a.x + k * (F::Q ? 1u : 2u);
        if constexpr (F::Q) {
            const float s = X == ST_X_MXFP8 ? scale_of<ST_KIND_MXFP8>(in ? a.xs[k / 32] : 0) : 1.0f;
#pragma unroll
            for (int h = 0; h < E / 16; ++h) {
                u32x4 c = {0, 0, 0, 0};
                if (all) c = *reinterpret_cast<const u32x4_any*>(px + 16 * h);
                else if (in) c = load_chunk(px + 16 * h, int64_t(a.k) - (k + 16 * h));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const u32x4 t = codes8<false, ST_KIND_MXFP8>(c[2 * i], c[2 * i + 1], s);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[8 * h + 4 * i + j] = t[j];
                }
            }
        } else {
#pragma unroll
            for (int h = 0; h < E / 8; ++h) {
                u32x4 c = {0, 0, 0, 0}, lo;
                if (all) c = *reinterpret_cast<const u32x4_any*>(px + 16 * h);
                else if (in) c = load_chunk(px + 16 * h, 2 * (int64_t(a.k) - (k + 8 * h)));
                if constexpr (D::SPLIT) split_f16(c, c, lo);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[4 * h + j] = c[j];
                    if constexpr (D::SPLIT) xl[4 * h + j] = lo[j];
                }
            }
        }
        float f = 0.0f;                    // the lane's fp32 scale, where the kinds have one per 128 of K
        if constexpr (F::GROUPED) {
            if (in) f = reinterpret_cast<const float*>(a.ws)[uint64_t(n0 / 128) * groups + k / 128];
            if (X == ST_X_FP8_GROUP128 && in) f *= reinterpret_cast<const float*>(a.xs)[k / 128];
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            // 16 elements at a time: an NVFP4 block, half an MX block
            float part = 0.0f;
#pragma unroll
            for (int b = 0; b < E / 16; ++b) {
                u32x4 v[2];
                const float s = is_mx(WK) ? scale_of<WK>(ws[r]) : 1.0f;
                if constexpr (WK == ST_KIND_NVFP4) {
                    // the codes alone (exact in bf16 and fp16): the block's sum takes the scale
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (D::F16) {
                            v[h][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[r][2 * b + h], 1.0f, 0));
                            v[h][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[r][2 * b + h], 1.0f, 1));
                            v[h][2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[r][2 * b + h], 1.0f, 2));
                            v[h][3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[r][2 * b + h], 1.0f, 3));
                        } else {
                            v[h] = codes8<false, ST_KIND_MXFP4>(w[r][2 * b + h], 0, 1.0f);
                        }
                    }
                } else if constexpr (F::FP4) {
                    v[0] = codes8<D::F16, WK>(w[r][2 * b], 0, s);
                    v[1] = codes8<D::F16, WK>(w[r][2 * b + 1], 0, s);
                } else {
                    v[0] = codes8<D::F16, WK>(w[r].x, w[r].y, s);
                    v[1] = codes8<D::F16, WK>(w[r].z, w[r].w, s);
                }
                float d = WK == ST_KIND_NVFP4 ? 0.0f : part;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    d = dot2<D::F16>(v[i / 4][i % 4], x[8 * b + i], d);
                    if constexpr (D::SPLIT) d = dot2<false>(v[i / 4][i % 4], xl[8 * b + i], d);
                }
                if constexpr (WK == ST_KIND_NVFP4) acc[r] = __builtin_fmaf(d, scale_of<WK>(ws[r] >> (8 * b) & 0xFF), acc[r]);
                else part = d;
            }
            if constexpr (WK != ST_KIND_NVFP4) acc[r] = F::GROUPED ? __builtin_fmaf(part, f, acc[r]) : acc[r] + part;
        }
    }
    const float v = fold<R>(acc);
    if (lane < R) joined[wave][lane] = v;
    __syncthreads();
    if (threadIdx.x == 0) {                // the slices in their order
        f32x4 t = {0, 0, 0, 0};
        for (uint32_t o = 0; o < waves; ++o) t += *reinterpret_cast<const f32x4*>(joined[o]);
        finish<X, WK>(a, 0, n0, t);
    }
}

// ------------------------------------------------------------------------- few rows

// 1 < m <= 16: one 16x16x32 instruction takes all rows of x.  Bound by the weight's bytes and x's, which every workgroup reads from L2
// (block FP8 [12288, 4096], 8 rows: 16.0 us; 12.1 without reading x; reading the weight alone takes 11.5).  A wavefront holds a turn of K, 64 bytes of a weight row per lane,
// for NT groups of 16 weight rows, all of it in flight at once straight into registers, and reads its part of x once for them; the
// wavefronts of a workgroup take different turns of the same weight rows and join in LDS.
template <int X_, int WK_>
struct Few {
    static constexpr int X = X_, WK = WK_;
    static constexpr bool Q = is_q(X), FP4 = is_fp4(WK), GROUPED = WK == ST_KIND_FP8_BLOCK128;
    static constexpr int NT = few_groups(WK), WAVES = few_waves(WK);
    static constexpr int LK = FP4 ? 128 : 64;        // elements of K a lane takes per turn (64 bytes of the weight)
    static constexpr int SS = 4 * LK;                // elements of K per turn
    static constexpr int CK = LK / 4;                // elements per 16-byte chunk of the weight
    static constexpr int XE = Q ? 1 : 2;             // bytes per element of x
    static constexpr int XL = CK * XE / 16;          // 16-byte pieces of x that go with a weight chunk
    // scale bytes of a lane's elements
    static constexpr int WSB = WK == ST_KIND_NVFP4 ? LK / 16 : is_mx(WK) ? LK / 32 : 0;
    static constexpr int XSB = X == ST_X_MXFP8 ? LK / 32 : 0;
    // K of lane group q's chunk j: neighbouring chunks belong to one lane, so that its scales are adjacent; with a scale per 128
    // of K, chunk j of all lanes together is 64 of K instead, and a scale belongs to whole instructions.
    static __device__ __forceinline__ uint32_t k_of(uint32_t q, uint32_t j) { return GROUPED ? 64 * j + 16 * q : LK * q + CK * j; }
};

// BYTES scale codes at p; not WHOLE: `avail` of them lie in the row, the others are 0.
template <int BYTES, bool WHOLE>
__device__ __forceinline__ uint64_t load_scales(const uint8_t* p, int64_t avail) {
    if constexpr (BYTES == 0) return 0;
    else if constexpr (!WHOLE) return load_codes(p, avail, BYTES < 4 ? BYTES : 4) | (BYTES == 8 ? uint64_t(load_codes(p + 4, avail - 4, 4)) << 32 : 0);
    else if constexpr (BYTES == 8) return *reinterpret_cast<const u64_any*>(p);
    else if constexpr (BYTES == 4) return *reinterpret_cast<const u32_any*>(p);
    else return *reinterpret_cast<const u16_any*>(p);
}
template <bool WHOLE>
__device__ __forceinline__ u32x4 load_piece(const uint8_t* p, int64_t avail) {
    if constexpr (WHOLE) return *reinterpret_cast<const u32x4_any*>(p);
    else return load_chunk(p, avail);
}

template <bool V>
struct Flag {
    static constexpr bool value = V;
};

template <class F>
__global__ __launch_bounds__(64 * F::WAVES) void linear_few(Args a) {
    constexpr int X = F::X, WK = F::WK, NT = F::NT;
    using D = Dense<X, WK>;
    __shared__ __align__(16) float joined[F::WAVES][NT][256];
    const int lane = threadIdx.x & 63, row = lane & 15, q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const uint32_t n0 = blockIdx.x * (16 * NT);
    const bool have = uint32_t(row) < a.m;        // lanes of rows that are not there load nothing: their column of D is not stored
    const uint32_t xrow = have ? row : 0;
    const uint32_t w_row = F::FP4 ? a.k / 2 : a.k, ws_row = a.k / (WK == ST_KIND_NVFP4 ? 16 : 32);
    const uint32_t groups = (a.k + 127) / 128;
    const uint8_t* px = a.x + xrow * a.x_pitch * F::XE;
    f32x4 acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = f32x4{0, 0, 0, 0};

    // a turn: K from k0; WHOLE: all SS elements are there, else there are zeros behind the end
    auto turn = [&](uint32_t k0, auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        const uint32_t kq = k0 + F::LK * q;        // K of this lane's scales
        u32x4 w[NT][4], xr[4][F::XL];
        uint64_t wsc[NT], xsc = 0;
        float gs[F::GROUPED ? NT : 1][2];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < F::XL; ++h) xr[j][h] = u32x4{0, 0, 0, 0};
        if (have) {
            if constexpr (F::XSB != 0) xsc = load_scales<F::XSB, WHOLE>(a.xs + xrow * uint64_t(a.k / 32) + kq / 32, int64_t(a.k / 32) - kq / 32);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t k = k0 + F::k_of(q, j);
#pragma unroll
                for (int h = 0; h < F::XL; ++h)
                    xr[j][h] = load_piece<WHOLE>(px + k * F::XE + 16 * h, (int64_t(a.k) - k) * F::XE - 16 * h);
            }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const uint32_t r = n0 + i * 16 + row, at = r < a.n ? r : a.n - 1;
            const uint8_t* pw = a.w + uint64_t(at) * w_row;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t k = k0 + F::k_of(q, j);
                const uint32_t to = F::FP4 ? k / 2 : k;
                w[i][j] = load_piece<WHOLE>(pw + to, int64_t(w_row) - to);
            }
            if constexpr (F::WSB != 0) {
                const uint32_t to = kq / (WK == ST_KIND_NVFP4 ? 16 : 32);
                wsc[i] = load_scales<F::WSB, WHOLE>(a.ws + uint64_t(at) * ws_row + to, int64_t(ws_row) - to);
            }
            if constexpr (F::GROUPED) {
                const uint32_t nb = (n0 + i * 16) / 128, lastb = (a.n - 1) / 128;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const uint32_t kb = k0 / 128 + g < groups ? k0 / 128 + g : groups - 1;
                    gs[i][g] = reinterpret_cast<const float*>(a.ws)[uint64_t(nb < lastb ? nb : lastb) * groups + kb];
                    if constexpr (X == ST_X_FP8_GROUP128) gs[i][g] *= reinterpret_cast<const float*>(a.xs)[uint64_t(xrow) * groups + kb];
                }
            }
        }
        u32x4 xv[4][F::CK / 8], xl[D::SPLIT ? 4 : 1][D::SPLIT ? F::CK / 8 : 1];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < F::XL; ++h) {
                const u32x4 c = xr[j][h];
                if constexpr (F::Q) {
                    const float s = X == ST_X_MXFP8 ? scale_of<ST_KIND_MXFP8>(uint32_t(xsc >> (8 * (j * F::CK / 32))) & 0xFF) : 1.0f;
                    xv[j][2 * h] = codes8<false, ST_KIND_MXFP8>(c.x, c.y, s);
                    xv[j][2 * h + 1] = codes8<false, ST_KIND_MXFP8>(c.z, c.w, s);
                } else if constexpr (D::SPLIT) {
                    split_f16(c, xv[j][h], xl[j][h]);
                } else {
                    xv[j][h] = c;
                }
            }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            f32x4 c = acc[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (F::GROUPED && (j & 1) == 0) c = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int h = 0; h < F::CK / 8; ++h) {
                    u32x4 wv;
                    if constexpr (WK == ST_KIND_NVFP4) {
                        wv = codes8<D::F16, WK>(w[i][j][h], 0, scale_of<WK>(uint32_t(wsc[i] >> (8 * (2 * j + h / 2))) & 0xFF));
                    } else if constexpr (F::FP4) {
                        wv = codes8<D::F16, WK>(w[i][j][h], 0, scale_of<WK>(uint32_t(wsc[i] >> (8 * j)) & 0xFF));
                    } else {
                        const float s = F::WSB ? scale_of<WK>(uint32_t(wsc[F::WSB ? i : 0] >> (8 * (j / 2))) & 0xFF) : 1.0f;
                        wv = codes8<D::F16, WK>(w[i][j][2 * h], w[i][j][2 * h + 1], s);
                    }
                    c = mfma32<D::F16>(wv, xv[j][h], c);
                    if constexpr (D::SPLIT) c = mfma32<false>(wv, xl[j][h], c);
                }
                // a group behind K's end has a sum of 0 and must not meet the last group's scale, which may be infinite
                if (F::GROUPED && (j & 1) == 1 && (WHOLE || k0 + 64 * (j - 1) < a.k)) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][r] = __builtin_fmaf(c[r], gs[F::GROUPED ? i : 0][j / 2], acc[i][r]);
                }
            }
            if constexpr (!F::GROUPED) acc[i] = c;
        }
    };
    // K is split over blockIdx.y too: a.steps turns each
    const uint32_t begin = blockIdx.y * a.steps * F::SS;
    const uint32_t end = a.k - begin < a.steps * F::SS ? a.k : begin + a.steps * F::SS;
    for (uint32_t k0 = begin + wave * F::SS; k0 < end; k0 += waves * F::SS) {
        if (k0 + F::SS <= a.k) turn(k0, Flag<true>{});
        else turn(k0, Flag<false>{});
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4*>(&joined[wave][i][lane * 4]) = acc[i];
    __syncthreads();
    // lane l of the first NT wavefronts adds up its four sums, in the order of the wavefronts
    for (uint32_t i = wave; i < NT; i += waves) {
        f32x4 v = *reinterpret_cast<const f32x4*>(&joined[0][i][lane * 4]);
        for (uint32_t o = 1; o < waves; ++o) v += *reinterpret_cast<const f32x4*>(&joined[o][i][lane * 4]);
        emit<X, WK>(a, blockIdx.y, row, n0 + i * 16 + 4 * q, v);
    }
}

// ------------------------------------------------------------------------- tiles

// What bounds it: 8-bit rows, tiles of 256: the matrix instructions (MXFP8 [12288, 4096] x 8192 rows: 476 us, of which they are busy
// 164; LDS reads take 90, the rest is waiting at the barrier and for LDS at a step's start).  Dense rows, tiles of 128: matrix
// instructions, decoding and LDS reads count 215, 125 and 220 us of NVFP4 [25600, 5120] x 2048 rows' 560-575 us and overlap in part.
//
// A tile of BM x BN outputs by WAVES_M x WAVES_N wavefronts; a step of K is 128 bytes of x: 64 elements, or 128
// of e4m3.  LDS holds rows of 16-byte chunks; chunk c of row r sits at c ^ swizzle(r), so that eight lanes
// reading the same chunk of eight consecutive rows touch all 32 banks once.
// F8 (8-bit x): the f8f6f4 matrix instructions, at twice the bf16 rate; otherwise both sides are widened to bf16.
template <int X_, int WK_, int BM_, int BN_, int WAVES_M_, int WAVES_N_, bool F8_, int STAGES_>
struct Tile {
    static constexpr int STAGES = STAGES_;
    static constexpr int X = X_, WK = WK_, BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
    static constexpr bool Q = is_q(X), FP4 = is_fp4(WK), F8 = F8_;
    static constexpr int THREADS = 64 * WAVES_M * WAVES_N;
    static constexpr int KS = Q ? 128 : 64;
    static constexpr int XB = 128, WB = KS / (FP4 ? 2 : 1);       // bytes of a row per step
    static constexpr int XC = XB / 16, WC = WB / 16;               // chunks of a row
    static constexpr int MT = BM / WAVES_M / 16, NT = BN / WAVES_N / 16;
    // scale bytes of a row per step (0: none) and elements per scale
    static constexpr int WSB = WK == ST_KIND_NVFP4 ? KS / 16 : is_mx(WK) ? KS / 32 : 0;
    static constexpr int XSB = X == ST_X_MXFP8 || X == ST_X_FP8_GROUP128 ? 4 : 0;
    static constexpr bool GROUPED = WK == ST_KIND_FP8_BLOCK128;    // sums scaled per 128 of K
    // wavefronts that load the scale words of the tile's x rows and weight rows (a word a row and step) in the direct modes
    static constexpr int X_WAVES = XSB ? BM / 64 : 0, W_WAVES = WSB ? BN / 64 : 0;
    static constexpr int STAGE = BM * XB + BN * WB + (XSB ? BM * 4 : 0) + (WSB ? BN * 4 : 0);
    static constexpr int X_PER = BM * XC / THREADS, W_PER = (BN * WC + THREADS - 1) / THREADS;
    static_assert(BM * XC % THREADS == 0 && BM <= THREADS && BN <= THREADS, "tile");
    static_assert(!GROUPED || (BN / WAVES_N <= 64 && BN % 64 == 0), "a wavefront's columns lie in one scale block");
    static __device__ __forceinline__ int x_at(int r, int c) { return r * XB + ((c ^ (r & 7)) << 4); }
    static __device__ __forceinline__ int w_at(int r, int c) {
        return r * WB + ((c ^ ((r / (8 / WC)) & (WC - 1))) << 4);
    }
};

// How a step's bytes reach LDS.  WHOLE: K is whole steps and every row starts on 16 bytes (scale words on 4), so they go there
// straight from global memory, STAGES - 1 steps on their way.  TAIL: rows start and end on 16 bytes; as WHOLE, except that a
// last, partial step (zeros behind the rows' ends) and the scale words of blocks pass through registers.  ANY: all of it passes through
// registers, one step ahead.  2000 bf16 rows through FP8 [5000, K]: K 4992 WHOLE 104 us, K 5008 TAIL 128 (ANY 162), K 5003 ANY 196;
// through MXFP8 with MXFP8 rows: K 4992 WHOLE 93, K 5024 TAIL 129 (ANY 210).
enum Path { ANY, TAIL, WHOLE };
// s_waitcnt for vmcnt(n) and lgkmcnt(0), expcnt at its maximum (gfx9 encoding: vmcnt in bits 3:0 and 15:14)
constexpr int wait_vmem(int n) { return (n & 15) | (n >> 4) << 14 | 7 << 4; }
// A wave-uniform fp32 that the kernel never writes, by the scalar unit.
__device__ __forceinline__ float ld_uniform_f32(const uint8_t* p) {
    return *reinterpret_cast<const __attribute__((address_space(4))) float*>(reinterpret_cast<uintptr_t>(p));
}
constexpr int kRawBufferWord3 = 0x00020000;  // V# word 3 of an untyped buffer (32-bit data format)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const uint8_t* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, 0x7FFFFFFF, kRawBufferWord3);
}
// 16 bytes per lane from base + voff + soff to LDS at `to` + 16 * lane; `to` is the same for the wavefront.
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t base, uint8_t* to, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(base, (__attribute__((address_space(3))) void*)to, 16, int(voff), int(soff), 0, 0);
}

template <class T, Path PATH>
__global__ __launch_bounds__(T::THREADS, 2) void linear_tile(Args a) {
    constexpr int X = T::X, WK = T::WK, MT = T::MT, NT = T::NT;
    constexpr bool DIRECT = PATH != ANY;
    // scale words straight to LDS: a group's fp32 are whole words in every row
    constexpr bool SCALES = T::X_WAVES + T::W_WAVES != 0, WORDS = SCALES && (PATH == WHOLE || (DIRECT && X == ST_X_FP8_GROUP128));
    constexpr int S = DIRECT ? T::STAGES : 2;
    __shared__ __align__(128) uint8_t lds[S][T::STAGE];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int row = lane & 15, q = lane >> 4;
    const int wm = wave / T::WAVES_N, wn = wave % T::WAVES_N;

    // Workgroup b runs on XCD b mod 8: renumber so that each XCD takes consecutive tiles, and order tiles in
    // bands of 8 row tiles so that neighbours share rows of both sides in that XCD's L2.
    const uint32_t total = a.tiles_m * a.tiles_n;
    uint32_t b = blockIdx.x;
    {
        const uint32_t per = total / 8, extra = total % 8, xcd = b % 8, at = b / 8;
        b = xcd * per + (xcd < extra ? xcd : extra) + at;
    }
    const uint32_t band = b / (8 * a.tiles_n), in = b - band * 8 * a.tiles_n;
    const uint32_t rows = a.tiles_m - band * 8 < 8 ? a.tiles_m - band * 8 : 8;
    const uint32_t m0 = (band * 8 + in % rows) * T::BM, n0 = in / rows * T::BN;
    const uint32_t split = blockIdx.y;
    const uint32_t all = (a.k + T::KS - 1) / T::KS;
    const uint32_t first = split * a.steps, last = first + a.steps < all ? first + a.steps : all;

    const uint64_t x_row = a.x_pitch * (T::Q ? 1 : 2), w_row = T::FP4 ? a.k / 2 : a.k;
    const uint64_t x_len = uint64_t(a.k) * (T::Q ? 1 : 2);
    const uint64_t ws_row = a.k / (WK == ST_KIND_NVFP4 ? 16 : 32);
    const uint32_t groups = (a.k + 127) / 128;
    // rows past the last are read as the last one; nothing of them is stored
    auto xr = [&](uint32_t r) { return m0 + r < a.m ? m0 + r : a.m - 1; };
    auto wr = [&](uint32_t r) { return n0 + r < a.n ? n0 + r : a.n - 1; };

    // Offsets from the tile's first row, the step's offset added by the scalar unit.  DIRECT loads take 32-bit ones (the host
    // sends rows too far apart for them the other way) and swap chunks on the way, since their place in LDS is fixed; the others
    // swap when they write LDS.
    using Off = std::conditional_t<DIRECT, uint32_t, uint64_t>;
    const __amdgpu_buffer_rsrc_t bx = rows_at(a.x + m0 * x_row), bw = rows_at(a.w + n0 * w_row);
    Off x_off[T::X_PER], w_off[T::W_PER];
#pragma unroll
    for (int i = 0; i < T::X_PER; ++i) {
        const int s = i * T::THREADS + tid, r = s / T::XC, c = (s % T::XC) ^ (DIRECT ? r & 7 : 0);
        x_off[i] = Off(xr(r) - m0) * Off(x_row) + c * 16;
    }
#pragma unroll
    for (int i = 0; i < T::W_PER; ++i) {
        const int s = i * T::THREADS + tid, r = s / T::WC, c = (s % T::WC) ^ (DIRECT ? (r / (8 / T::WC)) & (T::WC - 1) : 0);
        w_off[i] = s < T::BN * T::WC ? Off(wr(r) - n0) * Off(w_row) + c * 16 : 0;
    }
    const uint64_t xs_row = X == ST_X_MXFP8 ? a.k / 32 : 4ull * groups;
    const int uwave = __builtin_amdgcn_readfirstlane(wave);
    const bool x_scales = uwave < T::X_WAVES;
    const uint8_t* scales = x_scales ? a.xs + m0 * xs_row : a.ws + n0 * ws_row;
    const __amdgpu_buffer_rsrc_t bs = rows_at(scales);
    Off s_off = 0;
    if constexpr (SCALES)
        s_off = x_scales ? Off(xr(tid) - m0) * Off(xs_row) : Off(wr(tid - T::X_WAVES * 64) - n0) * Off(ws_row);
    u32x4 rx[DIRECT ? 1 : T::X_PER], rw[DIRECT ? 1 : T::W_PER];      // chunks on their way through registers
    uint32_t word = 0;                                               // and a row's scales

    auto issue = [&](uint32_t step, int buf) {
        const uint64_t kb = uint64_t(step) * T::XB, wb = uint64_t(step) * T::WB;
        uint8_t* sx = lds[buf];
        uint8_t* sw = lds[buf] + T::BM * T::XB;
        const bool whole = uint64_t(step + 1) * T::KS <= a.k;
        if constexpr (SCALES && !WORDS) {
            if (uwave < T::X_WAVES + T::W_WAVES) {
                const uint32_t bytes = x_scales ? T::XSB : T::WSB, at = step * bytes;
                const uint8_t* p = scales + at + s_off;
                if (!whole && !(X == ST_X_FP8_GROUP128 && x_scales))
                    word = load_codes(p, int64_t(x_scales ? xs_row : ws_row) - at, bytes);
                else if (bytes == 4) word = *reinterpret_cast<const u32_any*>(p);
                else word = *reinterpret_cast<const u16_any*>(p);
            }
        }
        if (DIRECT && (PATH == WHOLE || whole)) {
#pragma unroll
            for (int i = 0; i < T::X_PER; ++i)
                to_lds(bx, sx + (i * T::THREADS + wave * 64) * 16, x_off[i], uint32_t(kb));
#pragma unroll
            for (int i = 0; i < T::W_PER; ++i)
                if (T::BN * T::WC % T::THREADS == 0 || i * T::THREADS + uwave * 64 < T::BN * T::WC)
                    to_lds(bw, sw + (i * T::THREADS + wave * 64) * 16, w_off[i], uint32_t(wb));
        } else if constexpr (PATH == TAIL) {
            // once per tile: a loop that keeps the registers of the others free
#pragma unroll 1
            for (int s = tid; s < T::BM * T::XC; s += T::THREADS) {
                const int r = s / T::XC, c = (s % T::XC) ^ (r & 7);
                u32x4 v = {0, 0, 0, 0};
                if (kb + c * 16 < x_len) v = *reinterpret_cast<const u32x4*>(a.x + xr(r) * x_row + kb + c * 16);
                *reinterpret_cast<u32x4*>(sx + s * 16) = v;
            }
#pragma unroll 1
            for (int s = tid; s < T::BN * T::WC; s += T::THREADS) {
                const int r = s / T::WC, c = (s % T::WC) ^ ((r / (8 / T::WC)) & (T::WC - 1));
                u32x4 v = {0, 0, 0, 0};
                if (wb + c * 16 < w_row) v = *reinterpret_cast<const u32x4*>(a.w + wr(r) * w_row + wb + c * 16);
                *reinterpret_cast<u32x4*>(sw + s * 16) = v;
            }
            // a wavefront with no chunk of this step has loaded nothing, which the loop's counts do not know
            __builtin_amdgcn_s_waitcnt(wait_vmem(0));
        } else if constexpr (PATH == ANY) {
            const uint8_t* px = a.x + m0 * x_row + kb;
            const uint8_t* pw = a.w + n0 * w_row + wb;
            if (whole) {
#pragma unroll
                for (int i = 0; i < T::X_PER; ++i) rx[i] = *reinterpret_cast<const u32x4_any*>(px + x_off[i]);
#pragma unroll
                for (int i = 0; i < T::W_PER; ++i) rw[i] = *reinterpret_cast<const u32x4_any*>(pw + w_off[i]);
            } else {
#pragma unroll
                for (int i = 0; i < T::X_PER; ++i)
                    rx[i] = load_chunk(px + x_off[i], int64_t(x_len) - int64_t(kb + (i * T::THREADS + tid) % T::XC * 16));
#pragma unroll
                for (int i = 0; i < T::W_PER; ++i)
                    rw[i] = load_chunk(pw + w_off[i], int64_t(w_row) - int64_t(wb + (i * T::THREADS + tid) % T::WC * 16));
            }
        }
        if constexpr (WORDS) {
            if (uwave < T::X_WAVES + T::W_WAVES)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    bs, (__attribute__((address_space(3))) void*)(sw + T::BN * T::WB + wave * 256), 4, int(s_off),
                    int(T::WSB == 2 ? step / 2 * 4 : step * 4), 0, 0);
        }
    };
    // What issue() left in registers goes to LDS.
    auto commit = [&](int buf) {
        uint8_t* sx = lds[buf];
        uint8_t* sw = lds[buf] + T::BM * T::XB;
        if constexpr (PATH == ANY) {
#pragma unroll
            for (int i = 0; i < T::X_PER; ++i) {
                const int s = i * T::THREADS + tid;
                *reinterpret_cast<u32x4*>(sx + T::x_at(s / T::XC, s % T::XC)) = rx[i];
            }
#pragma unroll
            for (int i = 0; i < T::W_PER; ++i) {
                const int s = i * T::THREADS + tid;
                if (s < T::BN * T::WC) *reinterpret_cast<u32x4*>(sw + T::w_at(s / T::WC, s % T::WC)) = rw[i];
            }
        }
        if constexpr (SCALES && !WORDS) {
            if (uwave < T::X_WAVES + T::W_WAVES) reinterpret_cast<uint32_t*>(sw + T::BN * T::WB)[tid] = word;
        }
    };

    f32x4 acc[NT][MT], part[T::GROUPED && !T::F8 ? NT : 1][T::GROUPED && !T::F8 ? MT : 1];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    // loads of a step that this wavefront issues: BASE, one more with weight chunks left over, one more with scale words
    constexpr int BASE = T::X_PER + T::BN * T::WC / T::THREADS;
    const int loads = BASE + (uwave * 64 < T::BN * T::WC % T::THREADS ? 1 : 0) + (WORDS && uwave < T::X_WAVES + T::W_WAVES ? 1 : 0);
    const uint32_t count = last > first ? last - first : 0;
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
        if (uint32_t(i) < count) {
            issue(first + i, i);
            commit(i);
        }
    int buf = 0;
    for (uint32_t i = 0; i < count; ++i) {
        const uint32_t step = first + i;
        // This step's bytes are in LDS, and no wavefront reads the buffer that is filled next any more.  The loads of the S - 2
        // steps behind this one may still be on their way (they end in the order they were issued).
        if constexpr (DIRECT) {
            if (S == 2 || count - i <= S - 2) __builtin_amdgcn_s_waitcnt(wait_vmem(0));
            else if (loads == BASE) __builtin_amdgcn_s_waitcnt(wait_vmem((S - 2) * BASE));
            else if (loads == BASE + 1) __builtin_amdgcn_s_waitcnt(wait_vmem((S - 2) * (BASE + 1)));
            else __builtin_amdgcn_s_waitcnt(wait_vmem((S - 2) * (BASE + 2)));
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "singlethread");
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "singlethread");
        } else {
            __syncthreads();
        }
        const int fill = buf + S - 1 < S ? buf + S - 1 : buf - 1;
        if (i + S - 1 < count) issue(step + S - 1, fill);
        const uint8_t* sx = lds[buf];
        const uint8_t* sw = sx + T::BM * T::XB;
        const uint8_t* sxs = sw + T::BN * T::WB;
        const uint8_t* sws = sxs + (T::XSB ? T::BM * 4 : 0);
        float gs = 0.0f;       // the weight's scale of this wavefront's columns and this group of K
        if constexpr (T::GROUPED) {
            const uint32_t nb = (n0 + wn * (NT * 16)) / 128, lastb = (a.n - 1) / 128;
            // a scalar load: a vector load would wait for the steps on their way
            const uint32_t gi = __builtin_amdgcn_readfirstlane((nb < lastb ? nb : lastb) * groups + step * T::KS / 128);
            gs = ld_uniform_f32(a.ws + 4ull * gi);
        }
        if constexpr (!T::F8) {
            using D = Dense<X, WK>;
            // 64 of K at a time: lane group q holds 16q..16q+15 of them, 8 for each of two instructions
#pragma unroll
            for (int h = 0; h < T::KS / 64; ++h) {
                // the weight's operands stay, x's pass by
                u32x4 wv[NT][2];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int r = (wn * NT + i) * 16 + row;
                    const float s = T::WSB ? scale_of<WK>(sws[r * 4 + (WK == ST_KIND_NVFP4 ? q : 2 * (T::WSB == 2 ? (PATH == WHOLE ? step & 1 : 0) : h) + (q >> 1))]) : 1.0f;
                    if constexpr (T::FP4) {
                        const u32x2 c = *reinterpret_cast<const u32x2*>(sw + T::w_at(r, 2 * h + (q >> 1)) + (q & 1) * 8);
                        wv[i][0] = codes8<D::F16, WK>(c.x, 0, s);
                        wv[i][1] = codes8<D::F16, WK>(c.y, 0, s);
                    } else {
                        const u32x4 c = *reinterpret_cast<const u32x4*>(sw + T::w_at(r, q + 4 * h));
                        wv[i][0] = codes8<D::F16, WK>(c.x, c.y, s);
                        wv[i][1] = codes8<D::F16, WK>(c.z, c.w, s);
                    }
                }
                // GROUPED: sums of 128 of K start at zero and are scaled into acc at the end
                const bool begin = T::GROUPED && (T::Q ? h == 0 : (step & 1) == 0 || step == first);
                const bool end = T::GROUPED && (T::Q ? h == 1 : (step & 1) == 1 || i + 1 == count);
                // x's operands of the next 16 rows are on their way from LDS while these multiply
                u32x4 raw[2];
                uint32_t code = 0;
                auto next = [&](int j) {
                    const int r = (wm * MT + j) * 16 + row;
                    raw[0] = *reinterpret_cast<const u32x4*>(sx + T::x_at(r, T::Q ? q + 4 * h : 2 * q));
                    if constexpr (!T::Q) raw[1] = *reinterpret_cast<const u32x4*>(sx + T::x_at(r, 2 * q + 1));
                    if constexpr (X == ST_X_MXFP8) code = sxs[r * 4 + 2 * h + (q >> 1)];
                };
                next(0);
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    u32x4 xv[2], xl[2];
                    if constexpr (T::Q) {
                        const float s = X == ST_X_MXFP8 ? scale_of<ST_KIND_MXFP8>(code) : 1.0f;
                        xv[0] = codes8<false, ST_KIND_MXFP8>(raw[0].x, raw[0].y, s);
                        xv[1] = codes8<false, ST_KIND_MXFP8>(raw[0].z, raw[0].w, s);
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            xv[i] = raw[i];
                            if constexpr (D::SPLIT) split_f16(raw[i], xv[i], xl[i]);
                        }
                    }
                    if (j + 1 < MT) next(j + 1);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        f32x4 c = T::GROUPED ? (begin ? f32x4{0, 0, 0, 0} : part[T::GROUPED ? i : 0][T::GROUPED ? j : 0]) : acc[i][j];
                        c = mfma32<D::F16>(wv[i][0], xv[0], c);
                        c = mfma32<D::F16>(wv[i][1], xv[1], c);
                        if constexpr (D::SPLIT) {
                            c = mfma32<false>(wv[i][0], xl[0], c);
                            c = mfma32<false>(wv[i][1], xl[1], c);
                        }
                        if constexpr (T::GROUPED) part[i][j] = c;
                        else acc[i][j] = c;
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                if constexpr (T::GROUPED) {
                    if (end) {
#pragma unroll
                        for (int j = 0; j < MT; ++j) {
                            float f = gs;
                            if constexpr (X == ST_X_FP8_GROUP128)
                                f *= reinterpret_cast<const float*>(sxs)[(wm * MT + j) * 16 + row];
#pragma unroll
                            for (int i = 0; i < NT; ++i)
#pragma unroll
                                for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(part[i][j][r], f, acc[i][j][r]);
                        }
                    }
                }
            }
        } else {
            // k of lane group q in a 16x16x128 operand: e4m3 16q..16q+15 and 64+16q..64+16q+15, e2m1 32q..32q+31;
            // the scale of lane group q belongs to 32q..32q+31
            i32x8 wv[NT];
            int we[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int r = (wn * NT + i) * 16 + row;
                const u32x4 lo = *reinterpret_cast<const u32x4*>(sw + T::w_at(r, q));
                if constexpr (T::FP4) {
                    wv[i] = i32x8{int(lo.x), int(lo.y), int(lo.z), int(lo.w), 0, 0, 0, 0};
                } else {
                    const u32x4 hi = *reinterpret_cast<const u32x4*>(sw + T::w_at(r, q + 4));
                    wv[i] = i32x8{int(lo.x), int(lo.y), int(lo.z), int(lo.w), int(hi.x), int(hi.y), int(hi.z), int(hi.w)};
                }
                we[i] = T::WSB ? sws[r * 4 + q] : 127;
            }
            // x's operand of the next 16 rows is on its way from LDS while this one multiplies
            i32x8 xn;
            int en = 127;
            float fn = 0.0f;
            auto next = [&](int j) {
                const int r = (wm * MT + j) * 16 + row;
                const u32x4 lo = *reinterpret_cast<const u32x4*>(sx + T::x_at(r, q));
                const u32x4 hi = *reinterpret_cast<const u32x4*>(sx + T::x_at(r, q + 4));
                xn = i32x8{int(lo.x), int(lo.y), int(lo.z), int(lo.w), int(hi.x), int(hi.y), int(hi.z), int(hi.w)};
                if constexpr (X == ST_X_MXFP8) en = sxs[r * 4 + q];
                if constexpr (T::GROUPED) fn = reinterpret_cast<const float*>(sxs)[r];
            };
            next(0);
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                const i32x8 xv = xn;
                const int xe = en;
                const float xf = fn * gs;
                if (j + 1 < MT) next(j + 1);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    if constexpr (T::GROUPED) {
                        const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv[i], xv, f32x4{0, 0, 0, 0}, 0, 0, 0, 127, 0, 127);
#pragma unroll
                        for (int t = 0; t < 4; ++t) acc[i][j][t] = __builtin_fmaf(p[t], xf, acc[i][j][t]);
                    } else {
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv[i], xv, acc[i][j], T::FP4 ? 4 : 0, 0, 0, we[i], 0, xe);
                    }
                }
            }
        }
        if (i + S - 1 < count) commit(fill);
        buf = buf + 1 < S ? buf + 1 : 0;
    }
    // Two 16-row groups at a time go through LDS, so that a row's columns are stored together and the epilogue's code, with its
    // choices of type and activation, is there once per two groups (unrolled over all of them it outgrew the instruction cache:
    // 760 us became 2740 for 8192 rows through MXFP8 [12288, 4096] in tiles of 256).
    constexpr int PITCH = NT * 16 + 4, PER = 64 / (NT * 4);      // floats of a row in LDS; rows a wavefront stores together
    static_assert(T::WAVES_M * T::WAVES_N * 32 * PITCH * 4 <= 2 * T::STAGE, "the epilogue's rows fit the stages' LDS");
    float* mine = reinterpret_cast<float*>(&lds[0][0]) + wave * 32 * PITCH;
    __syncthreads();
#pragma unroll
    for (int j0 = 0; j0 < MT; j0 += 2) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < NT; ++i)
                *reinterpret_cast<f32x4*>(mine + (j * 16 + row) * PITCH + i * 16 + 4 * q) = acc[i][j0 + j];
#pragma unroll 1
        for (int r = lane / (NT * 4); r < 32; r += PER) {
            const int c = lane % (NT * 4) * 4;
            const f32x4 v = *reinterpret_cast<const f32x4*>(mine + r * PITCH + c);
            emit<X, WK>(a, split, m0 + (wm * MT + j0) * 16 + r, n0 + wn * (NT * 16) + c, v);
        }
    }
}

// ------------------------------------------------------------------------- launches

template <class T, bool LARGE>
void launch_tile(const Args& a, const Plan& p, hipStream_t s) {
    const dim3 grid(a.tiles_m * a.tiles_n, a.splits), block(T::THREADS);
    if (p.direct && !p.tail) hipLaunchKernelGGL((linear_tile<T, WHOLE>), grid, block, 0, s, a);
    if constexpr (!LARGE || !is_mx(T::WK))
        if (p.direct && p.tail) hipLaunchKernelGGL((linear_tile<T, TAIL>), grid, block, 0, s, a);
    if constexpr (!LARGE)
        if (!p.direct) hipLaunchKernelGGL((linear_tile<T, ANY>), grid, block, 0, s, a);
}

template <int X, int WK>
void launch(const Args& a, const Plan& p, hipStream_t s) {
    if (p.one) {
        hipLaunchKernelGGL((linear_one<One<X, WK>>), dim3((a.n + One<X, WK>::R - 1) / One<X, WK>::R), dim3(64 * p.waves), 0, s, a);
        return;
    }
    if (p.few) {
        const dim3 grid((a.n + 16 * Few<X, WK>::NT - 1) / (16 * Few<X, WK>::NT), a.splits), block(64 * p.waves);
        hipLaunchKernelGGL((linear_few<Few<X, WK>>), grid, block, 0, s, a);
    } else if (p.bm == 64) {
        launch_tile<Tile<X, WK, 64, 64, 2, 2, false, 4>, false>(a, p, s);
    } else if (p.bm == 128) {
        if constexpr (is_q(X))
            if (p.f8) launch_tile<Tile<X, WK, 128, 128, 2, 2, true, 2>, false>(a, p, s);
        // Packed fp4 under dense rows: a wavefront takes all rows of the tile, so that each code is decoded once (NVFP4 [25600, 5120]
        // x 2048 rows: 574 us against 625 with a quadrant each, in turn); the 8-bit kinds, cheaper to decode, read less LDS in quadrants.
        if (!is_q(X) || !p.f8) launch_tile<Tile<X, WK, 128, 128, is_fp4(WK) && !is_q(X) ? 1 : 2, is_fp4(WK) && !is_q(X) ? 4 : 2, false, 2>, false>(a, p, s);
    } else if constexpr (is_q(X)) {
        launch_tile<Tile<X, WK, 256, 256, 2, 4, true, 2>, true>(a, p, s);
    }
    if (a.part) {
        const uint64_t items = uint64_t((a.n + 3) / 4) * a.m;
        hipLaunchKernelGGL((linear_join<X, WK>), dim3(uint32_t((items + 255) / 256)), dim3(256), 0, s, a);
    }
}

}  // namespace
}  // namespace st_linear_impl
