// The experts of a mixture on their stored weights:
//   h[p] = act(gate_e x_t) * (up_e x_t)   for each pair p = (t, j) of a token and its j-th expert e
//   y[t] = sum_j weights[t, j] down_e h[t, j] + residual[t]
// Weights enter as st_linear's do (linear_kernels.h: exact codes times scales, fp32 sums).  h is kept as two bf16 terms, 16 significant bits with
// bf16's range: one term would add as much again to a bf16 result's own rounding, and more than that to an fp16 one's.
//
// Bound by the bytes of the chosen experts' weights; x and h, few rows, come from L2.  No atomics on results: every sum has its order.
//  * one token: up_one, down_one, dot products on the vector unit at the rate the weights arrive; a lane has 16 bytes of a row, and in
//    down_one the lanes go through all experts' rows as if they were one.
//  * few pairs of an expert: up_few, a workgroup for 16 rows of gate and of up of an expert, its wavefronts taking different parts of K.
//  * up to 16 tokens with few pairs in all: down_few, a workgroup for 16 or 32 columns of y, its wavefronts taking all experts' parts of K in turn.
//    The columns of its instructions are the tokens, so that the sum over experts is the sum over K and needs no second pass.
//  * else: tiles of 64 pairs of one expert by 64 rows of gate and of up, or 128 of down; x or h staged through LDS for four wavefronts, weights
//    straight to their registers; down's results of the pairs pass through memory and `combine` adds them.
// (moe.cpp has the borders.)
#pragma once

#include "linear_kernels.h"
#include "moe.h"

namespace st_moe_impl {
namespace {

using namespace st_dev;
using st_linear_impl::Dense;
using st_linear_impl::dot2;
using st_linear_impl::fold;
using st_linear_impl::load_scales;

// How rows meet the weight: as they are, fp16 split in two bf16 terms, or two terms in memory.
enum Rows { PLAIN, SPLIT, TWO };

// The 16 bytes at p, of which `avail` belong to a row of `row` bytes, the others 0.  Where the row ends among them they come from a load
// that ends with the row, shifted.
__device__ __forceinline__ u32x4 load_end(const uint8_t* p, int32_t avail, uint32_t row) {
    u32x4 v = {0, 0, 0, 0};
    if (avail >= 16) {
        v = *reinterpret_cast<const u32x4_any*>(p);
    } else if (avail > 0 && row >= 16) {
        const uint32_t back = 16 - uint32_t(avail), by = back & 3;
        v = *reinterpret_cast<const u32x4_any*>(p - back);
        if (back & 4) v = u32x4{v[1], v[2], v[3], 0};
        if (back & 8) v = u32x4{v[2], v[3], 0, 0};
        v = u32x4{__builtin_amdgcn_alignbyte(v[1], v[0], by), __builtin_amdgcn_alignbyte(v[2], v[1], by),
                  __builtin_amdgcn_alignbyte(v[3], v[2], by), __builtin_amdgcn_alignbyte(0, v[3], by)};
    } else {
        uint64_t lo = 0, hi = 0;
#pragma unroll 1
        for (int i = 0; i < int(avail); ++i) (i < 8 ? lo : hi) |= uint64_t(p[i]) << (8 * (i & 7));
        v = u32x4{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
    }
    return v;
}
// How a turn ends: within K; at K's end, which cuts no 16 bytes of a weight's row; or anywhere (kernels of their own, since the shifted
// loads take twice the registers).
enum Ends { WITHIN, EVEN, ODD };
// (avail is 32 bits of something the compiler knows nothing of: it would keep each load's own in a register through the loop)
__device__ __forceinline__ int32_t bytes_left(int64_t v) {
    int32_t n = v < -1024 ? -1024 : v > 4096 ? 4096 : int32_t(v);
    asm volatile("" : "+v"(n));
    return n;
}
template <Ends END>
__device__ __forceinline__ u32x4 load_piece(const uint8_t* p, int32_t avail, uint32_t row) {
    if constexpr (END == WITHIN) return *reinterpret_cast<const u32x4_any*>(p);
    else if constexpr (END == EVEN) return avail > 0 ? u32x4(*reinterpret_cast<const u32x4_any*>(p)) : u32x4{0, 0, 0, 0};
    else return load_end(p, avail, row);
}
template <Ends END>
struct Ending {
    static constexpr Ends value = END;
};

// A row's data and scales of one matrix of an expert, in a uniform form.
struct Matrix {
    const uint8_t *w, *s, *s2;
};
__device__ __forceinline__ Matrix matrix_of(const Args& a, uint32_t expert, int which) {
    // (an address from memory may point anywhere for the compiler, which would take flat loads: these are global memory)
    typedef const __attribute__((address_space(1))) uint8_t* global;
    const st_moe_weight& m = a.experts_dev[uint64_t(expert) * 3 + which];
    auto at = [](const void* p) { return (const uint8_t*)(global)reinterpret_cast<uintptr_t>(p); };
    return Matrix{at(m.w), at(m.scale), at(m.scale2)};
}
template <int WK>
__device__ __forceinline__ float tensor_scale(const Matrix& m) {
    if constexpr (WK == ST_KIND_FP8_TENSOR) return *reinterpret_cast<const float*>(m.s);
    else if constexpr (WK == ST_KIND_NVFP4) return *reinterpret_cast<const float*>(m.s2);
    else return 1.0f;
}

// A turn of K for a wavefront: 256 elements, 64 per lane group.
template <int WK>
struct Turn {
    static constexpr bool FP4 = is_fp4(WK), GROUPED = WK == ST_KIND_FP8_BLOCK128;
    static constexpr int SS = 256, LK = 64;
    static constexpr int CHUNKS = FP4 ? 2 : 4, CK = LK / CHUNKS;      // 16-byte chunks of a weight row per lane, elements of one
    static constexpr int WSB = WK == ST_KIND_NVFP4 ? LK / 16 : is_mx(WK) ? LK / 32 : 0;
    // Neighbouring chunks belong to one lane, so that its scales are adjacent; with a scale per 128 of K, chunk j of all lanes together is
    // 64 of K instead, and a scale belongs to whole instructions.
    static __device__ __forceinline__ uint32_t k_of(uint32_t q, uint32_t j) { return GROUPED ? 64 * j + 16 * q : LK * q + CK * j; }
};

// The codes and scales of a turn from k0 for NG groups of 16 weight rows; n[i]: this lane's row.  Zeros behind K's end.
template <int WK, int NG>
struct Codes {
    using F = Turn<WK>;
    u32x4 w[NG][F::CHUNKS];
    uint32_t sc[NG];
    float gs[NG][2];

    template <Ends END>
    __device__ __forceinline__ void load(const Matrix (&mat)[NG], const uint32_t (&n)[NG], uint32_t k0, uint32_t K) {
        const int q = (threadIdx.x & 63) >> 4;
        const uint32_t w_row = F::FP4 ? K / 2 : K, ws_row = K / (WK == ST_KIND_NVFP4 ? 16 : 32), groups = (K + 127) / 128;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const uint32_t to = (k0 + F::k_of(q, 0)) / (F::FP4 ? 2 : 1);
            const uint8_t* pw = mat[i].w + uint64_t(n[i]) * w_row + to;
            const int32_t left = END == WITHIN ? 0 : bytes_left(int64_t(w_row) - to);
#pragma unroll
            for (int j = 0; j < F::CHUNKS; ++j) {
                constexpr int STEP = F::GROUPED ? 64 : 16;      // bytes between a lane's chunks
                w[i][j] = load_piece<END>(pw + STEP * j, left - STEP * j, w_row);
            }
            if constexpr (F::WSB != 0) {
                const uint32_t to = (k0 + F::LK * q) / (WK == ST_KIND_NVFP4 ? 16 : 32);
                sc[i] = uint32_t(load_scales<F::WSB, END == WITHIN>(mat[i].s + uint64_t(n[i]) * ws_row + to, int64_t(ws_row) - to));
            }
            if constexpr (F::GROUPED) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const uint32_t kb = k0 / 128 + g < groups ? k0 / 128 + g : groups - 1;
                    gs[i][g] = reinterpret_cast<const float*>(mat[i].s)[uint64_t(n[i] / 128) * groups + kb];
                }
            }
        }
    }
    // acc += the products with this lane's row at px (its second term at pl), with the scales of blocks.  Lanes that do not `have` a row load
    // nothing, their columns are 0 (40 fp16 tokens through MXFP4, 6 pairs an expert: 74 us, 83 when they load another's row).
    // (PARTS of x at a time, which bounds the registers it takes)
    template <bool F16, Rows R, Ends END, int PARTS>
    __device__ __forceinline__ void times(const uint8_t* px, const uint8_t* pl, uint32_t k0, uint32_t K, f32x4 (&acc)[NG], bool have) const {
        const int q = (threadIdx.x & 63) >> 4;
        constexpr int XL = F::CK / 8;
        constexpr int HALF = F::CHUNKS / PARTS;
        static_assert(PARTS == 1 || PARTS == 2, "a group of 128 is half a turn");
        const uint64_t to = uint64_t(k0 + F::k_of(q, 0)) * 2;
        const int32_t left = END == WITHIN ? 0 : bytes_left(int64_t(K) * 2 - int64_t(to));
#pragma unroll
        for (int half = 0; half < PARTS; ++half) {
            u32x4 xr[HALF][XL], xl[R == PLAIN ? 1 : HALF][XL];
#pragma unroll
            for (int j = 0; j < HALF; ++j)
#pragma unroll
                for (int h = 0; h < XL; ++h) {
                    xr[j][h] = u32x4{0, 0, 0, 0};
                    if constexpr (R != PLAIN) xl[j][h] = u32x4{0, 0, 0, 0};
                }
            if (have) {
#pragma unroll
                for (int j = 0; j < HALF; ++j)
#pragma unroll
                    for (int h = 0; h < XL; ++h) {
                        const int at = 2 * (F::GROUPED ? 64 : F::CK) * (half * HALF + j) + 16 * h;
                        xr[j][h] = load_piece<END>(px + to + at, left - at, 2 * K);
                        if constexpr (R == TWO) xl[j][h] = load_piece<END>(pl + to + at, left - at, 2 * K);
                        if constexpr (R == SPLIT) split_f16(xr[j][h], xr[j][h], xl[j][h]);
                    }
            }
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                f32x4 c = F::GROUPED ? f32x4{0, 0, 0, 0} : acc[i];
#pragma unroll
                for (int b = 0; b < HALF; ++b) {
                    const int j = half * HALF + b;
#pragma unroll
                    for (int h = 0; h < XL; ++h) {
                        u32x4 wv;
                        if constexpr (WK == ST_KIND_NVFP4) wv = codes8<F16, WK>(w[i][j][h], 0, scale_of<WK>(sc[i] >> (8 * (2 * j + h / 2)) & 0xFF));
                        else if constexpr (F::FP4) wv = codes8<F16, WK>(w[i][j][h], 0, scale_of<WK>(sc[i] >> (8 * j) & 0xFF));
                        else wv = codes8<F16, WK>(w[i][j][2 * h], w[i][j][2 * h + 1], F::WSB ? scale_of<WK>(sc[i] >> (8 * (j / 2)) & 0xFF) : 1.0f);
                        c = mfma32<F16>(wv, xr[b][h], c);
                        if constexpr (R != PLAIN) c = mfma32<F16>(wv, xl[b][h], c);
                    }
                    // a group of 128 behind K's end has a sum of 0 and must not meet the last group's scale, which may be infinite
                    if (F::GROUPED && (j & 1) == 1) {
                        if (END == WITHIN || k0 + 64 * (j - 1) < K) {
#pragma unroll
                            for (int r = 0; r < 4; ++r) acc[i][r] = __builtin_fmaf(c[r], gs[i][j / 2], acc[i][r]);
                        }
                        c = f32x4{0, 0, 0, 0};
                    }
                }
                if constexpr (!F::GROUPED) acc[i] = c;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};

// h as two terms, each to be rounded to bf16; infinities and NaN stay whole in the first.  It is cut, not rounded, where rounding would make an infinity of a
// number between bf16's largest and fp32's.
__device__ __forceinline__ void terms_of(float h, float& hi, float& lo) {
    const uint32_t rounded = cvt_bf16x2(h, 0.0f) << 16, cut = as_u32(h) & 0xFFFF0000u;
    hi = as_f32((rounded & 0x7FFFFFFFu) == 0x7F800000u ? cut : rounded);
    const float rest = h - hi;
    lo = rest == rest ? rest : 0.0f;
}
// h of columns n..n+3 of pair p, from the sums of gate and up.
template <int WK>
__device__ __forceinline__ void store_h(const Args& a, uint32_t p, uint32_t n, f32x4 gate, f32x4 up, float sg, float su) {
    if (n >= a.i) return;
    float hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) terms_of(activate(gate[i] * sg, a.act) * (up[i] * su), hi[i], lo[i]);
    // (h_pitch is a multiple of 8, so columns behind the last one have room)
    uint8_t* at = a.h + (uint64_t(p) * a.h_pitch + n) * 2;
    *reinterpret_cast<dword2*>(at) = dword2{cvt_bf16x2(hi[0], hi[1]), cvt_bf16x2(hi[2], hi[3])};
    *reinterpret_cast<dword2*>(at + uint64_t(a.pairs) * a.h_pitch * 2) = dword2{cvt_bf16x2(lo[0], lo[1]), cvt_bf16x2(lo[2], lo[3])};
}

// Columns n..n+3 of token t.
__device__ __forceinline__ void store_y(const Args& a, uint32_t t, uint32_t n, f32x4 v) {
    if (n >= a.n) return;
    const uint32_t cnt = a.n - n < 4 ? a.n - n : 4;
    float y[4] = {v[0], v[1], v[2], v[3]};
    const uint64_t o = uint64_t(t) * a.out_pitch + n, r = uint64_t(t) * a.res_pitch + n;
    if (a.vec && cnt == 4) {
        if (a.res) {
            float w[4];
            load4_as_f32(a.res, a.res_type, r, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] += w[i];
        }
        store4(a.out, a.out_type, o, y);
    } else {
        for (uint32_t i = 0; i < cnt; ++i) {
            if (a.res) y[i] += load_as_f32(a.res, a.res_type, r + i);
            store_as(a.out, a.out_type, o + i, y[i]);
        }
    }
}

// The k-th expert that has pairs and its part of the sorted list; no pairs: there is none.
struct Entry {
    uint32_t expert, count;
    const uint32_t* pairs;
};
__device__ __forceinline__ Entry entry_of(const Args& a, uint32_t k) {
    if (k >= a.sorted[0]) return Entry{0, 0, nullptr};
    const uint32_t* e = a.sorted + 4 + 4 * k;
    return Entry{e[0], e[2], a.sorted + 4 + 4 * a.slots + e[1]};
}

// ------------------------------------------------------------------------- one token

// As linear_one (linear_kernels.h).  A lane's 16 bytes of a weight row hold E elements of K; its part of x stays in registers for R rows.
template <int WK>
struct One {
    static constexpr bool FP4 = is_fp4(WK), GROUPED = WK == ST_KIND_FP8_BLOCK128;
    static constexpr int E = FP4 ? 32 : 16;
};
// One row's 16 bytes and scale codes from element k of K; zeros behind its end.
template <int WK>
__device__ __forceinline__ void load_row(const uint8_t* pw, const uint8_t* ps, uint32_t k, uint32_t K, u32x4& w, uint32_t& sc) {
    using O = One<WK>;
    const uint32_t at = O::FP4 ? k / 2 : k, row = O::FP4 ? K / 2 : K;
    w = u32x4{0, 0, 0, 0};
    sc = 0;
    if (k + O::E <= K) {
        w = *reinterpret_cast<const u32x4_any*>(pw + at);
        if constexpr (WK == ST_KIND_NVFP4) sc = *reinterpret_cast<const u16_any*>(ps + k / 16);
    } else if (k < K) {
        w = load_end(pw + at, bytes_left(int64_t(row) - at), row);
        if constexpr (WK == ST_KIND_NVFP4) sc = ps[k / 16];
    }
    if constexpr (is_mx(WK)) sc = k < K ? ps[k / 32] : 0;
}
// Its products with E elements of a row in one or two terms, the scales of blocks of 16 and 32 applied.
template <int WK, bool F16, bool TERMS>
__device__ __forceinline__ float dot_row(u32x4 w, uint32_t sc, const uint32_t* x, const uint32_t* xl) {
    using O = One<WK>;
    float sum = 0.0f;
#pragma unroll
    for (int b = 0; b < O::E / 16; ++b) {
        u32x4 v[2];
        const float s = is_mx(WK) ? scale_of<WK>(sc) : 1.0f;
        if constexpr (WK == ST_KIND_NVFP4) {
            // the codes alone (exact in bf16 and fp16): the block's sum takes the scale
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (F16) {
                    v[h][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[2 * b + h], 1.0f, 0));
                    v[h][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[2 * b + h], 1.0f, 1));
                    v[h][2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[2 * b + h], 1.0f, 2));
                    v[h][3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[2 * b + h], 1.0f, 3));
                } else {
                    v[h] = codes8<false, ST_KIND_MXFP4>(w[2 * b + h], 0, 1.0f);
                }
            }
        } else if constexpr (O::FP4) {
            v[0] = codes8<F16, WK>(w[2 * b], 0, s);
            v[1] = codes8<F16, WK>(w[2 * b + 1], 0, s);
        } else {
            v[0] = codes8<F16, WK>(w.x, w.y, s);
            v[1] = codes8<F16, WK>(w.z, w.w, s);
        }
        float d = WK == ST_KIND_NVFP4 ? 0.0f : sum;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            d = dot2<F16>(v[i / 4][i % 4], x[8 * b + i], d);
            if constexpr (TERMS) d = dot2<F16>(v[i / 4][i % 4], xl[8 * b + i], d);
        }
        if constexpr (WK == ST_KIND_NVFP4) sum = __builtin_fmaf(d, scale_of<WK>(sc >> (8 * b) & 0xFF), sum);
        else sum = d;
    }
    return sum;
}
// E elements of a bf16 or fp16 row from element k of K as pairs, zeros behind its end.
template <int E>
__device__ __forceinline__ void load_pairs(const uint8_t* p, uint32_t k, uint32_t K, uint32_t* x) {
#pragma unroll
    for (int h = 0; h < E / 8; ++h) {
        const uint32_t at = k + 8 * h;
        u32x4 c = {0, 0, 0, 0};
        if (k + E <= K) c = *reinterpret_cast<const u32x4_any*>(p + uint64_t(at) * 2);
        else if (at < K) c = load_end(p + uint64_t(at) * 2, bytes_left((int64_t(K) - at) * 2), 2 * K);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * h + j] = c[j];
    }
}

// Columns of a workgroup (packed-fp4 experts [1280, 5120], 8 of them: gate and up 17 us with two, 21 with four, 31 with eight; down 15 us with
// two, 12 with four).
constexpr int kOneMaxWaves = 8, kUpColumns = 2, kDownColumns = 4;

// kUpColumns columns of h of pair blockIdx.y: their rows of gate and of up.
template <int X, int WK>
__global__ __launch_bounds__(64 * kOneMaxWaves) void up_one(Args a) {
    using O = One<WK>;
    using D = Dense<X, WK>;
    constexpr int R = 2 * kUpColumns, PAIRS = O::E / 2;
    __shared__ __align__(16) float joined[kOneMaxWaves][R];
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int32_t e = __builtin_amdgcn_readfirstlane(a.ids[blockIdx.y]);
    if (e < 0 || uint32_t(e) >= a.experts) return;
    const Matrix mat[2] = {matrix_of(a, e, 0), matrix_of(a, e, 1)};
    const uint32_t n0 = blockIdx.x * kUpColumns, w_row = O::FP4 ? a.k / 2 : a.k, ws_row = a.k / (WK == ST_KIND_NVFP4 ? 16 : 32);
    const uint32_t groups = (a.k + 127) / 128;
    float acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = 0.0f;
    for (uint32_t k0 = wave * 64 * O::E; k0 < a.k; k0 += waves * 64 * O::E) {
        const uint32_t k = k0 + lane * O::E;
        u32x4 w[R];
        uint32_t sc[R];
        // rows past the last are read as the last one; nothing of them is stored
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t n = n0 + r % kUpColumns < a.i ? n0 + r % kUpColumns : a.i - 1;
            const Matrix& m = mat[r / kUpColumns];
            load_row<WK>(m.w + uint64_t(n) * w_row, m.s + uint64_t(n) * ws_row, k, a.k, w[r], sc[r]);
        }
        uint32_t x[PAIRS], xl[D::SPLIT ? PAIRS : 1];
        load_pairs<O::E>(a.x, k, a.k, x);
        if constexpr (D::SPLIT) {
#pragma unroll
            for (int h = 0; h < PAIRS / 4; ++h) {
                u32x4 hi, lo;
                split_f16(u32x4{x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]}, hi, lo);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[4 * h + j] = hi[j], xl[4 * h + j] = lo[j];
            }
        }
        float f[2] = {1.0f, 1.0f};          // the lane's fp32 scales, where the kinds have one per 128 of K
        if constexpr (O::GROUPED) {
#pragma unroll
            for (int i = 0; i < 2; ++i) f[i] = k < a.k ? reinterpret_cast<const float*>(mat[i].s)[uint64_t(n0 / 128) * groups + k / 128] : 0.0f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float d = dot_row<WK, D::F16, D::SPLIT>(w[r], sc[r], x, xl);
            acc[r] = O::GROUPED ? __builtin_fmaf(d, f[r / kUpColumns], acc[r]) : acc[r] + d;
        }
    }
    const float v = fold<R>(acc);
    if (lane < R) joined[wave][lane] = v;
    __syncthreads();
    if (threadIdx.x < kUpColumns && n0 + threadIdx.x < a.i) {      // the slices in their order
        float g = 0.0f, up = 0.0f;
        for (uint32_t o = 0; o < waves; ++o) g += joined[o][threadIdx.x], up += joined[o][kUpColumns + threadIdx.x];
        float hi, lo;
        terms_of(activate(g * tensor_scale<WK>(mat[0]), a.act) * (up * tensor_scale<WK>(mat[1])), hi, lo);
        uint16_t* at = reinterpret_cast<uint16_t*>(a.h) + uint64_t(blockIdx.y) * a.h_pitch + n0 + threadIdx.x;
        at[0] = uint16_t(cvt_bf16x2(hi, 0.0f));
        at[uint64_t(a.pairs) * a.h_pitch] = uint16_t(cvt_bf16x2(lo, 0.0f));
    }
}

// kDownColumns columns of y: lane c of all the workgroup's lanes has chunks c, c + threads, ... of the pairs' rows, one after the
// other; its products take its own pair's weight and scales, and the sum over lanes is the sum over pairs.
template <int WK>
__global__ __launch_bounds__(64 * kOneMaxWaves) void down_one(Args a) {
    using O = One<WK>;
    constexpr int R = kDownColumns, PAIRS = O::E / 2;
    __shared__ __align__(16) float joined[kOneMaxWaves][R];
    const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const uint32_t n0 = blockIdx.x * R, w_row = O::FP4 ? a.i / 2 : a.i, ws_row = a.i / (WK == ST_KIND_NVFP4 ? 16 : 32), groups = (a.i + 127) / 128;
    const uint32_t chunks = (a.i + O::E - 1) / O::E;
    const uint64_t plane = uint64_t(a.pairs) * a.h_pitch * 2;
    float acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = 0.0f;
    for (uint32_t c = threadIdx.x; c < a.pairs * chunks; c += blockDim.x) {
        const uint32_t p = c / chunks, k = c % chunks * O::E;
        const int32_t e = a.ids[p];
        if (e < 0 || uint32_t(e) >= a.experts) continue;
        const Matrix m = matrix_of(a, e, 2);
        u32x4 w[R];
        uint32_t sc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t n = n0 + r < a.n ? n0 + r : a.n - 1;
            load_row<WK>(m.w + uint64_t(n) * w_row, m.s + uint64_t(n) * ws_row, k, a.i, w[r], sc[r]);
        }
        uint32_t x[PAIRS], xl[PAIRS];
        const uint8_t* ph = a.h + uint64_t(p) * a.h_pitch * 2;
        load_pairs<O::E>(ph, k, a.i, x);
        load_pairs<O::E>(ph + plane, k, a.i, xl);
        float f = a.weights[p] * tensor_scale<WK>(m);
        if constexpr (O::GROUPED) f *= reinterpret_cast<const float*>(m.s)[uint64_t(n0 / 128) * groups + k / 128];
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = __builtin_fmaf(dot_row<WK, false, true>(w[r], sc[r], x, xl), f, acc[r]);
    }
    const float v = fold<R>(acc);
    if (lane < R) joined[wave][lane] = v;
    __syncthreads();
    if (threadIdx.x < R && n0 + threadIdx.x < a.n) {
        const uint32_t n = n0 + threadIdx.x;
        float y = 0.0f;
        for (uint32_t o = 0; o < waves; ++o) y += joined[o][threadIdx.x];
        if (a.res) y += load_as_f32(a.res, a.res_type, n);
        store_as(a.out, a.out_type, n, y);
    }
}

// ------------------------------------------------------------------------- few pairs of an expert

// Bound by the weights' bytes: 8 tokens of 8 block-FP8 experts of 128 [1280, 4096] (39 to 47 different ones, 10.5 MB each) 83 us, 5 TB/s and more.  With
// fp16 rows through MXFP4 (40 tokens, 4 of 32 experts [1280, 5120], 24 or 25 different ones of 7 MB) by decoding: each row meets the weights as two bf16 terms, 74 us.
constexpr int kUpWaves = 4;

template <int X, int WK, Ends TAIL>
__global__ __launch_bounds__(64 * kUpWaves) void up_few(Args a) {
    using F = Turn<WK>;
    using D = Dense<X, WK>;
    constexpr Rows R = D::SPLIT ? SPLIT : PLAIN;
    __shared__ __align__(16) float joined[kUpWaves][2][256];
    const uint32_t lane = threadIdx.x & 63, row = lane & 15, q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const uint32_t n0 = blockIdx.x * 16;
    const Entry en = entry_of(a, blockIdx.y);
    if (en.count == 0) return;
    const Matrix mat[2] = {matrix_of(a, en.expert, 0), matrix_of(a, en.expert, 1)};
    const uint32_t at = n0 + row < a.i ? n0 + row : a.i - 1, n[2] = {at, at};
    // 16 pairs at a time; those of an expert that has more meet its weights again, from L2
    for (uint32_t c0 = 0; c0 < en.count; c0 += 16) {
        const bool have = c0 + row < en.count;
        const uint32_t p = en.pairs[have ? c0 + row : c0];
        const uint8_t* px = a.x + uint64_t(p / a.top) * a.x_pitch * 2;
        f32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        for (uint32_t k0 = wave * F::SS; k0 < a.k; k0 += waves * F::SS) {
            auto turn = [&](auto ending) {
                constexpr Ends END = decltype(ending)::value;
                Codes<WK, 2> codes;
                codes.template load<END>(mat, n, k0, a.k);
                codes.template times<D::F16, R, END, 2>(px, nullptr, k0, a.k, acc, have);
            };
            if (k0 + F::SS <= a.k) turn(Ending<WITHIN>{});
            else turn(Ending<TAIL>{});
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) *reinterpret_cast<f32x4*>(&joined[wave][i][lane * 4]) = acc[i];
        __syncthreads();
        if (wave == 0 && have) {
            f32x4 v[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[i] = *reinterpret_cast<const f32x4*>(&joined[0][i][lane * 4]);
                for (uint32_t o = 1; o < waves; ++o) v[i] += *reinterpret_cast<const f32x4*>(&joined[o][i][lane * 4]);
            }
            store_h<WK>(a, p, n0 + 4 * q, v[0], v[1], tensor_scale<WK>(mat[0]), tensor_scale<WK>(mat[1]));
        }
        __syncthreads();
    }
}

// 8 tokens of 8 experts of 128 (block FP8 [4096, 1280], 39 to 47 different ones, 5.2 MB each): 70 us, 3 TB/s and more.  Not for want of loads in flight (two
// turns' codes at once: the same); the two terms of h are four times the codes' bytes through the CU's cache.
// Entries: each expert that some token has; a second one for tokens that have it twice, and so on.
constexpr int kDownWaves = 16;
static_assert(kFewPairs == 64, "a lane for each pair");

template <int WK, int NG, Ends TAIL>
__global__ __launch_bounds__(64 * kDownWaves) void down_few(Args a) {
    using F = Turn<WK>;
    __shared__ __align__(16) float joined[kDownWaves][NG][256];
    __shared__ __align__(16) uint8_t pair_of[kFewPairs][16];      // an entry's pair of each token; kFewPairs: none
    __shared__ uint32_t expert[kFewPairs], number;
    const int lane = threadIdx.x & 63, row = lane & 15, q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t n0 = blockIdx.x * (16 * NG);
    if (wave == 0) {
        const uint32_t p = lane, j = p % a.top, none = kFewPairs * 0x01010101u;
        *reinterpret_cast<u32x4*>(pair_of[p]) = u32x4{none, none, none, none};
        const int32_t id = p < a.pairs ? a.ids[p] : -1;
        const bool valid = id >= 0 && uint32_t(id) < a.experts;
        uint32_t again = 0;
        for (uint32_t o = 0; o < a.top; ++o) again += __shfl(id, int(p - j + o)) == id && o < j ? 1 : 0;
        const uint32_t key = valid ? uint32_t(id) * kMaxTop + again : ~0u;
        uint32_t first = p;
        for (uint32_t o = 0; o < a.pairs; ++o) first = uint32_t(__builtin_amdgcn_readlane(int(key), int(o))) == key && o < first ? o : first;
        const uint64_t leaders = __ballot(valid && first == p);
        if (valid) {
            const uint32_t at = __popcll(leaders & ((uint64_t(1) << first) - 1));
            pair_of[at][p / a.top] = uint8_t(p);
            expert[at] = uint32_t(id);
        }
        if (lane == 0) number = __popcll(leaders);
    }
    __syncthreads();
    const uint32_t entries = number;

    uint32_t n[NG];
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        const uint32_t r = n0 + 16 * i + row;
        n[i] = r < a.n ? r : a.n - 1;
    }
    f32x4 sum[NG];
#pragma unroll
    for (int i = 0; i < NG; ++i) sum[i] = f32x4{0, 0, 0, 0};
    const uint32_t turns = (a.i + F::SS - 1) / F::SS, items = entries * turns;
    const uint64_t plane = uint64_t(a.pairs) * a.h_pitch * 2;
    for (uint32_t item = wave; item < items; item += kDownWaves) {
        const uint32_t en = item / turns, k0 = item % turns * F::SS;
        const uint32_t e = __builtin_amdgcn_readfirstlane(expert[en]), of = pair_of[en][row];
        const bool have = of < kFewPairs;
        const uint32_t pr = have ? of : 0;
        const float weight = a.weights[pr];
        const uint8_t* ph = a.h + uint64_t(pr) * a.h_pitch * 2;
        Matrix mat[NG];
        mat[0] = matrix_of(a, e, 2);
#pragma unroll
        for (int i = 1; i < NG; ++i) mat[i] = mat[0];
        f32x4 acc[NG];
#pragma unroll
        for (int i = 0; i < NG; ++i) acc[i] = f32x4{0, 0, 0, 0};
        auto turn = [&](auto ending) {
            constexpr Ends END = decltype(ending)::value;
            Codes<WK, NG> codes;
            codes.template load<END>(mat, n, k0, a.i);
            codes.template times<false, TWO, END, NG>(ph, ph + plane, k0, a.i, acc, have);
        };
        if (k0 + F::SS <= a.i) turn(Ending<WITHIN>{});
        else turn(Ending<TAIL>{});
        if (have) {
            const float f = weight * tensor_scale<WK>(mat[0]);
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) sum[i][r] = __builtin_fmaf(acc[i][r], f, sum[i][r]);
        }
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) *reinterpret_cast<f32x4*>(&joined[wave][i][lane * 4]) = sum[i];
    __syncthreads();
    if (wave < NG) {
        f32x4 v = *reinterpret_cast<const f32x4*>(&joined[0][wave][lane * 4]);
#pragma unroll
        for (int o = 1; o < kDownWaves; ++o) v += *reinterpret_cast<const f32x4*>(&joined[o][wave][lane * 4]);
        if (uint32_t(row) < a.t) store_y(a, row, n0 + 16 * wave + 4 * q, v);
    }
}

// ------------------------------------------------------------------------- tiles

constexpr int kTileRows = 64, kTileThreads = 256, kUpK = 128;
// Steps of K (40 tokens through MXFP4's down [5120, 1280]: 46 us with 128, 64 with 64; 320 through block FP8's [4096, 1280]: 237 and 223)
constexpr int down_k(int wk) { return is_fp4(wk) ? 128 : 64; }

// UP: 64 rows of gate and of up; else 128 rows of down.  320 tokens of 8 block-FP8 experts of 128 (20 pairs each) through [1280, 4096]: gate and up 367 us,
// 3.6 TB/s, down 223 us, 3 TB/s: loads are one step ahead of the products, and the registers of two steps would cost a workgroup of each CU.
template <int WK, bool F16, Rows R, bool UP, int TK, Ends TAIL>
__global__ __launch_bounds__(kTileThreads, R == TWO && TK == 128 ? 2 : 3) void tile(Args a) {
    constexpr bool FP4 = is_fp4(WK), MX = is_mx(WK), GROUPED = WK == ST_KIND_FP8_BLOCK128;
    constexpr int PLANES = R == PLAIN ? 1 : 2, MT = kTileRows / 16;
    static_assert(TK == 128 || (TK == 64 && !FP4), "16 bytes of a weight row, or twice as many, per lane and step");
    constexpr int WC = TK == 128 && !FP4 ? 2 : 1;                             // chunks of a weight row per lane and step
    constexpr int OPS = TK / 32;                                              // instructions of a step for 16 x 16 results
    constexpr int XC = TK / 8, PER = kTileRows * XC / kTileThreads;           // 16-byte chunks of a row of x per step; per thread and plane
    __shared__ __align__(16) uint8_t lds[2][PLANES][kTileRows * TK * 2];
    // chunk c of row r of a step sits at c ^ swizzle(r): 16 lanes reading one chunk of 16 rows touch all banks once
    auto place = [](uint32_t r, uint32_t c) { return (r * XC + (c ^ (XC == 16 ? r & 15 : r >> 1 & 7))) * 16; };
    const int tid = threadIdx.x, lane = tid & 63, row = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Entry en = entry_of(a, blockIdx.y);
    if (en.count == 0) return;
    const uint32_t e = en.expert;
    const uint32_t K = UP ? a.k : a.i, N = UP ? a.i : a.n;
    const uint32_t n0 = UP ? blockIdx.x * 64 + wave * 16 : blockIdx.x * 128 + wave * 32;
    Matrix mat[2];
    mat[0] = matrix_of(a, e, UP ? 0 : 2);
    mat[1] = UP ? matrix_of(a, e, 1) : mat[0];
    uint32_t n[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t r = n0 + (UP ? 0 : 16 * i) + row;
        n[i] = r < N ? r : N - 1;
    }
    const uint32_t w_row = FP4 ? K / 2 : K, ws_row = K / (WK == ST_KIND_NVFP4 ? 16 : 32), groups = (K + 127) / 128, steps = (K + TK - 1) / TK;
    const uint64_t plane = uint64_t(a.pairs) * a.h_pitch * 2;

    for (uint32_t from = 0; from < en.count; from += kTileRows) {
        const uint32_t count = en.count - from < kTileRows ? en.count - from : kTileRows;
        const uint32_t* list = en.pairs + from;
        if (from) __syncthreads();
        const int mt = int(count + 15) / 16;
        const uint8_t* src[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t r = (i * kTileThreads + tid) / XC, p = list[r < count ? r : 0];
            src[i] = UP ? a.x + uint64_t(p / a.top) * a.x_pitch * 2 : a.h + uint64_t(p) * a.h_pitch * 2;
        }
        const uint32_t c = tid % XC;
        u32x4 rx[PLANES][PER], rw[2][WC];
        uint32_t rs[2][WC];
        float rg[2];
        auto load = [&](uint32_t step) {
            const uint32_t k0 = step * TK;
            const bool whole = k0 + TK <= K;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int j = 0; j < WC; ++j) {
                    const uint32_t k = k0 + (FP4 ? TK / 4 * q : 64 * j + 16 * q), to = FP4 ? k / 2 : k;
                    const uint8_t* p = mat[i].w + uint64_t(n[i]) * w_row + to;
                    rw[i][j] = whole ? load_piece<WITHIN>(p, 16, w_row) : load_piece<TAIL>(p, bytes_left(int64_t(w_row) - to), w_row);
                    if constexpr (WK == ST_KIND_NVFP4) {
                        const uint8_t* ps = mat[i].s + uint64_t(n[i]) * ws_row + k / 16;
                        rs[i][j] = whole ? *reinterpret_cast<const u16_any*>(ps) : load_codes(ps, int64_t(ws_row) - k / 16, 2);
                    } else if constexpr (MX) {
                        rs[i][j] = k < K ? mat[i].s[uint64_t(n[i]) * ws_row + k / 32] : 0;
                    }
                }
                if constexpr (GROUPED) rg[i] = reinterpret_cast<const float*>(mat[i].s)[uint64_t(n[i] / 128) * groups + step * TK / 128];
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if ((i * kTileThreads + tid) / XC >= uint32_t(16 * mt)) continue;
                const uint8_t* p = src[i] + (uint64_t(k0) + 8 * c) * 2;
                const int32_t avail = bytes_left((int64_t(K) - k0 - 8 * c) * 2);
                rx[0][i] = whole ? load_piece<WITHIN>(p, 16, 2 * K) : load_piece<TAIL>(p, avail, 2 * K);
                if constexpr (R == TWO) rx[1][i] = whole ? load_piece<WITHIN>(p + plane, 16, 2 * K) : load_piece<TAIL>(p + plane, avail, 2 * K);
            }
        };
        auto commit = [&](int buf) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint32_t r = (i * kTileThreads + tid) / XC;
                if (r >= uint32_t(16 * mt)) continue;
                if constexpr (R == SPLIT) split_f16(rx[0][i], rx[0][i], rx[1][i]);
#pragma unroll
                for (int p = 0; p < PLANES; ++p) *reinterpret_cast<u32x4*>(&lds[buf][p][place(r, c)]) = rx[p][i];
            }
        };
        f32x4 acc[2][MT];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
        if (steps) {
            load(0);
            commit(0);
        }
        for (uint32_t step = 0; step < steps; ++step) {
            // this step's weights to operands, each 32 of K: lane group q's eight elements are chunk `at` of x
            u32x4 wv[2][OPS];
            float gs[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                gs[i] = GROUPED ? rg[i] : 1.0f;
#pragma unroll
                for (int m = 0; m < OPS; ++m) {
                    if constexpr (WK == ST_KIND_NVFP4) wv[i][m] = codes8<F16, WK>(rw[i][0][m], 0, scale_of<WK>(rs[i][0] >> (8 * (m / 2)) & 0xFF));
                    else if constexpr (FP4) wv[i][m] = codes8<F16, WK>(rw[i][0][m], 0, scale_of<WK>(rs[i][0]));
                    else wv[i][m] = codes8<F16, WK>(rw[i][m / 2][2 * (m & 1)], rw[i][m / 2][2 * (m & 1) + 1], MX ? scale_of<WK>(rs[i][m / 2]) : 1.0f);
                }
            }
            __syncthreads();
            const int buf = step & 1;
            if (step + 1 < steps) load(step + 1);
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                if (j >= mt) continue;
                f32x4 v[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) v[i] = GROUPED ? f32x4{0, 0, 0, 0} : acc[i][j];
#pragma unroll
                for (int m = 0; m < OPS; ++m) {
                    const int at = FP4 ? OPS * q + m : 8 * (m / 2) + 2 * q + (m & 1);
#pragma unroll
                    for (int p = 0; p < PLANES; ++p) {
                        const u32x4 xv = *reinterpret_cast<const u32x4*>(&lds[buf][p][place(16 * j + row, at)]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) v[i] = mfma32<F16>(wv[i][m], xv, v[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = GROUPED ? __builtin_fmaf(v[i][r], gs[i], acc[i][j][r]) : v[i][r];
            }
            if (step + 1 < steps) commit(buf ^ 1);
        }
        const float s0 = tensor_scale<WK>(mat[0]), s1 = tensor_scale<WK>(mat[1]);
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            if (uint32_t(16 * j + row) >= count) continue;
            const uint32_t p = list[16 * j + row];
            if constexpr (UP) {
                store_h<WK>(a, p, n0 + 4 * q, acc[0][j], acc[1][j], s0, s1);
            } else {
                const float f = a.weights[p] * s0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t col = n0 + 16 * i + 4 * q;
                    float* o = a.part + uint64_t(p) * a.n + col;
                    const f32x4 v = acc[i][j] * f;
                    if ((a.n & 3) == 0 && col < a.n) *reinterpret_cast<f32x4*>(o) = v;
                    else
                        for (uint32_t r = 0; r < 4 && col + r < a.n; ++r) o[r] = v[r];
                }
            }
        }
    }
}

// go(kernel's Ends) for rows of K: those of the MX kinds always end on 16 bytes.
template <int WK, class F>
void by_end(uint32_t K, F go) {
    if constexpr (is_mx(WK)) return go(Ending<EVEN>{});
    else if ((is_fp4(WK) ? K / 2 : K) % 16 == 0) return go(Ending<EVEN>{});
    else return go(Ending<ODD>{});
}

// The gate and up products of rows of type X.
template <int X, int WK>
void launch_up(const Args& a, Cut cut, hipStream_t s) {
    using D = Dense<X, WK>;
    const uint32_t chunks = (a.k + One<WK>::E - 1) / One<WK>::E, turns = (a.k + Turn<WK>::SS - 1) / Turn<WK>::SS;
    const dim3 few((a.i + 15) / 16, a.slots), block(64 * even(turns, kUpWaves));
    by_end<WK>(a.k, [&](auto end) {
        constexpr Ends END = decltype(end)::value;
        switch (cut) {
            case ONE:
                hipLaunchKernelGGL((up_one<X, WK>), dim3((a.i + kUpColumns - 1) / kUpColumns, a.slots), dim3(64 * even((chunks + 63) / 64, kOneMaxWaves)), 0, s, a);
                break;
            case FEW:
            case SOME: hipLaunchKernelGGL((up_few<X, WK, END>), few, block, 0, s, a); break;
            case MANY:
                hipLaunchKernelGGL((tile<WK, D::F16, D::SPLIT ? SPLIT : PLAIN, true, kUpK, END>), dim3((a.i + 63) / 64, a.slots), dim3(kTileThreads), 0, s, a);
                break;
        }
    });
}

}  // namespace
}  // namespace st_moe_impl
