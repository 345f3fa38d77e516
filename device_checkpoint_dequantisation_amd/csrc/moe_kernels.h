// The experts of a mixture on their stored weights:
//   h[p] = act(gate_e x_t) * (up_e x_t)   for each pair p = (t, j) of a token and its j-th expert e
//   y[t] = sum_j weights[t, j] down_e h[t, j] + residual[t]
// Weights enter as st_linear's do (linear_kernels.h: exact codes times scales, fp32 sums).  h is kept as two bf16 terms, 16 significant bits with
// bf16's range: one term would add as much again to a bf16 result's own rounding, and more than that to an fp16 one's.
//
// Bound by the bytes of the chosen experts' weights; x and h, a few rows, come from L2.  No atomics: every sum has its order.
//  * few tokens (16): up_few, one workgroup for 16 rows of gate and up of an expert, its wavefronts taking different parts of K; down_few, one
//    workgroup for 16 or 32 columns of y, its wavefronts taking all experts' parts of K in turn, each instruction's 16 columns being the tokens, so
//    that the sum over experts is the sum over K and needs no second pass.
//  * more: tiles of 64 pairs of one expert by 64 rows of gate and of up, or 128 of down; x or h staged through LDS for four wavefronts, weights
//    straight to their registers; the pairs' results pass through memory and `combine` adds them.
#pragma once

#include "linear_kernels.h"
#include "moe.h"

namespace st_moe_impl {
namespace {

using namespace st_dev;
using st_linear_impl::Dense;
using st_linear_impl::Few;
using st_linear_impl::Flag;
using st_linear_impl::load_piece;
using st_linear_impl::load_scales;

// How rows meet the weight: as they are, fp16 split in two bf16 terms, or two terms in memory.
enum Rows { PLAIN, SPLIT, TWO };

// A row's data and scales of one matrix of an expert, in a uniform form.
struct Matrix {
    const uint8_t *w, *s, *s2;
};
__device__ __forceinline__ Matrix matrix_of(const Args& a, uint32_t expert, int which) {
    const st_moe_weight& m = a.experts_dev[uint64_t(expert) * 3 + which];
    return Matrix{static_cast<const uint8_t*>(m.w), static_cast<const uint8_t*>(m.scale), static_cast<const uint8_t*>(m.scale2)};
}
template <int WK>
__device__ __forceinline__ float tensor_scale(const Matrix& m) {
    if constexpr (WK == ST_KIND_FP8_TENSOR) return *reinterpret_cast<const float*>(m.s);
    else if constexpr (WK == ST_KIND_NVFP4) return *reinterpret_cast<const float*>(m.s2);
    else return 1.0f;
}

// A turn of K (Few::SS elements from k0) for NG groups of 16 weight rows: this lane's rows n[i], its row of x at px (and its second
// term at pl).  acc += the products, with the scales of blocks.  WHOLE: the turn lies within K, else there are zeros behind its end.
template <int WK, bool F16, Rows R, bool WHOLE, int NG>
__device__ __forceinline__ void turn(const Matrix (&mat)[NG], const uint32_t (&n)[NG], const uint8_t* px, const uint8_t* pl, bool have,
                                     uint32_t k0, uint32_t K, f32x4 (&acc)[NG]) {
    using F = Few<ST_X_BF16, WK>;
    const int q = (threadIdx.x & 63) >> 4;
    const uint32_t kq = k0 + F::LK * q, w_row = F::FP4 ? K / 2 : K, ws_row = K / (WK == ST_KIND_NVFP4 ? 16 : 32), groups = (K + 127) / 128;
    u32x4 w[NG][4], xr[4][F::XL], xl[R == PLAIN ? 1 : 4][F::XL];
    uint64_t wsc[NG];
    float gs[NG][2];
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        const uint8_t* pw = mat[i].w + uint64_t(n[i]) * w_row;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t k = k0 + F::k_of(q, j), to = F::FP4 ? k / 2 : k;
            w[i][j] = load_piece<WHOLE>(pw + to, int64_t(w_row) - to);
        }
        if constexpr (F::WSB != 0) {
            const uint32_t to = kq / (WK == ST_KIND_NVFP4 ? 16 : 32);
            wsc[i] = load_scales<F::WSB, WHOLE>(mat[i].s + uint64_t(n[i]) * ws_row + to, int64_t(ws_row) - to);
        }
        if constexpr (F::GROUPED) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const uint32_t kb = k0 / 128 + g < groups ? k0 / 128 + g : groups - 1;
                gs[i][g] = reinterpret_cast<const float*>(mat[i].s)[uint64_t(n[i] / 128) * groups + kb];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < F::XL; ++h) {
            xr[j][h] = u32x4{0, 0, 0, 0};
            if constexpr (R != PLAIN) xl[j][h] = u32x4{0, 0, 0, 0};
        }
    if (have) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < F::XL; ++h) {
                const uint32_t k = k0 + F::k_of(q, j) + 8 * h;
                xr[j][h] = load_piece<WHOLE>(px + uint64_t(k) * 2, (int64_t(K) - k) * 2);
                if constexpr (R == TWO) xl[j][h] = load_piece<WHOLE>(pl + uint64_t(k) * 2, (int64_t(K) - k) * 2);
                if constexpr (R == SPLIT) split_f16(xr[j][h], xr[j][h], xl[j][h]);
            }
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        f32x4 c = acc[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (F::GROUPED && (j & 1) == 0) c = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int h = 0; h < F::CK / 8; ++h) {
                u32x4 wv;
                if constexpr (WK == ST_KIND_NVFP4) {
                    wv = codes8<F16, WK>(w[i][j][h], 0, scale_of<WK>(uint32_t(wsc[i] >> (8 * (2 * j + h / 2))) & 0xFF));
                } else if constexpr (F::FP4) {
                    wv = codes8<F16, WK>(w[i][j][h], 0, scale_of<WK>(uint32_t(wsc[i] >> (8 * j)) & 0xFF));
                } else {
                    const float s = F::WSB ? scale_of<WK>(uint32_t(wsc[i] >> (8 * (j / 2))) & 0xFF) : 1.0f;
                    wv = codes8<F16, WK>(w[i][j][2 * h], w[i][j][2 * h + 1], s);
                }
                c = mfma32<F16>(wv, xr[j][h], c);
                if constexpr (R != PLAIN) c = mfma32<F16>(wv, xl[j][h], c);
            }
            // a group behind K's end has a sum of 0 and must not meet the last group's scale, which may be infinite
            if (F::GROUPED && (j & 1) == 1 && (WHOLE || k0 + 64 * (j - 1) < K)) {
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][r] = __builtin_fmaf(c[r], gs[i][j / 2], acc[i][r]);
            }
        }
        if constexpr (!F::GROUPED) acc[i] = c;
    }
}

// h of columns n..n+3 of pair p, from the sums of gate and up.
template <int WK>
__device__ __forceinline__ void store_h(const Args& a, uint32_t p, uint32_t n, f32x4 gate, f32x4 up, float sg, float su) {
    if (n >= a.i) return;
    float hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float h = activate(gate[i] * sg, a.act) * (up[i] * su);
        hi[i] = as_f32(cvt_bf16x2(h, 0.0f) << 16);
        const float rest = h - hi[i];
        lo[i] = rest == rest ? rest : 0.0f;      // infinities and NaN stay whole in the first term
    }
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

// The expert of this workgroup's slot, or -1.
__device__ __forceinline__ int32_t expert_of(const Args& a, uint32_t slot) {
    const int32_t e = a.by_pair ? a.ids[slot] : int32_t(slot);
    return e >= 0 && uint32_t(e) < a.experts ? __builtin_amdgcn_readfirstlane(e) : -1;
}

// ------------------------------------------------------------------------- up to 16 tokens

constexpr int up_waves(int wk) { return is_fp4(wk) ? 4 : 8; }

template <int X, int WK>
__global__ __launch_bounds__(64 * up_waves(WK)) void up_few(Args a) {
    using F = Few<ST_X_BF16, WK>;
    using D = Dense<X, WK>;
    constexpr Rows R = D::SPLIT ? SPLIT : PLAIN;
    __shared__ __align__(16) float joined[up_waves(WK)][2][256];
    __shared__ uint16_t list[kFewTokens * kMaxTop];
    __shared__ uint32_t found;
    const int lane = threadIdx.x & 63, row = lane & 15, q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const uint32_t n0 = blockIdx.x * 16, slot = blockIdx.y;
    const int32_t e = expert_of(a, slot);
    if (e < 0) return;
    if (wave == 0) {
        uint32_t count = 0;
        for (uint32_t p = 0; p < a.pairs; p += 64) {
            const bool mine = p + lane < a.pairs && a.ids[p + lane] == e;
            const uint64_t m = __ballot(mine);
            if (mine) list[count + __popcll(m & ((uint64_t(1) << lane) - 1))] = uint16_t(p + lane);
            count += __popcll(m);
        }
        if (lane == 0) found = count;
    }
    const Matrix mat[2] = {matrix_of(a, e, 0), matrix_of(a, e, 1)};
    __syncthreads();
    const uint32_t count = found;
    if (count == 0 || (a.by_pair && list[0] != slot)) return;
    const uint32_t at = n0 + row < a.i ? n0 + row : a.i - 1, n[2] = {at, at};
    for (uint32_t c0 = 0; c0 < count; c0 += 16) {
        const bool have = c0 + row < count;
        const uint32_t p = list[have ? c0 + row : c0];
        const uint8_t* px = a.x + uint64_t(p / a.top) * a.x_pitch * 2;
        f32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        for (uint32_t k0 = wave * F::SS; k0 < a.k; k0 += waves * F::SS) {
            if (k0 + F::SS <= a.k) turn<WK, D::F16, R, true, 2>(mat, n, px, nullptr, have, k0, a.k, acc);
            else turn<WK, D::F16, R, false, 2>(mat, n, px, nullptr, have, k0, a.k, acc);
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

// Entries: each expert that some token has; a second one for tokens that have it twice, and so on.  Row t of an entry is token t's pair, or none.
constexpr int kDownWaves = 8;
static_assert(kFewTokens * kMaxTop <= 64 * kDownWaves, "a thread for each pair");

template <int WK, int NG>
__global__ __launch_bounds__(64 * kDownWaves) void down_few(Args a) {
    using F = Few<ST_X_BF16, WK>;
    constexpr uint32_t MAX = kFewTokens * kMaxTop;
    constexpr uint16_t NONE = 0xFFFF;
    __shared__ __align__(16) float joined[kDownWaves][NG][256];
    __shared__ uint32_t key[MAX];
    __shared__ uint16_t entry[MAX], expert[MAX], pair[MAX][kFewTokens];
    __shared__ uint32_t leaders[kDownWaves];
    const int lane = threadIdx.x & 63, row = lane & 15, q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), p = threadIdx.x;
    const uint32_t n0 = blockIdx.x * (16 * NG);

    const int32_t id = p < a.pairs ? a.ids[p] : -1;
    const bool valid = id >= 0 && uint32_t(id) < a.experts;
    uint32_t mine = ~0u;
    if (valid) {
        uint32_t again = 0;
        for (uint32_t o = p / a.top * a.top; o < p; ++o) again += a.ids[o] == id ? 1 : 0;
        mine = uint32_t(id) * kMaxTop + again;
    }
    key[p] = mine;
    for (uint32_t i = p; i < MAX * kFewTokens / 2; i += 64 * kDownWaves) reinterpret_cast<uint32_t*>(pair)[i] = 0xFFFFFFFFu;
    __syncthreads();
    uint32_t first = p;
    for (uint32_t o = a.pairs; o-- > 0;)
        if (o < p && key[o] == mine) first = o;
    const bool leads = valid && first == p;
    const uint64_t m = __ballot(leads);
    if (lane == 0) leaders[wave] = __popcll(m);
    __syncthreads();
    uint32_t entries = 0, before = 0;
#pragma unroll
    for (uint32_t o = 0; o < kDownWaves; ++o) {
        before += o < wave ? leaders[o] : 0;
        entries += leaders[o];
    }
    if (leads) {
        const uint32_t at = before + __popcll(m & ((uint64_t(1) << lane) - 1));
        entry[p] = uint16_t(at);
        expert[at] = uint16_t(id);
    }
    __syncthreads();
    if (valid) pair[entry[first]][p / a.top] = uint16_t(p);
    __syncthreads();

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
        const uint32_t e = __builtin_amdgcn_readfirstlane(expert[en]);
        const uint16_t pr = pair[en][row];
        const bool have = pr != NONE;
        Matrix mat[NG];
        mat[0] = matrix_of(a, e, 2);
#pragma unroll
        for (int i = 1; i < NG; ++i) mat[i] = mat[0];
        const uint8_t* ph = a.h + uint64_t(have ? pr : 0) * a.h_pitch * 2;
        f32x4 acc[NG];
#pragma unroll
        for (int i = 0; i < NG; ++i) acc[i] = f32x4{0, 0, 0, 0};
        if (k0 + F::SS <= a.i) turn<WK, false, TWO, true, NG>(mat, n, ph, ph + plane, have, k0, a.i, acc);
        else turn<WK, false, TWO, false, NG>(mat, n, ph, ph + plane, have, k0, a.i, acc);
        if (have) {
            const float f = a.weights[pr] * tensor_scale<WK>(mat[0]);
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

// ------------------------------------------------------------------------- more tokens

constexpr int kTileRows = 64, kTileK = 128, kTileThreads = 256;

// The first pairs of expert e from `from` on, at most kTileRows, in their order: list, and their number.  All threads take part; ids are
// read 16 per thread at a time.
struct Found {
    uint32_t list[kTileRows];
    uint32_t sums[kTileThreads / 64];
};
__device__ __forceinline__ uint32_t find(const Args& a, int32_t e, uint32_t from, Found& f) {
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t count = 0;
    for (uint32_t base = from; base < a.pairs && count < kTileRows; base += 16 * kTileThreads) {
        const uint32_t p0 = base + tid * 16;
        uint32_t hits = 0;
        if (p0 + 16 <= a.pairs) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const u32x4 v = *reinterpret_cast<const u32x4_any*>(a.ids + p0 + 4 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) hits |= int32_t(v[i]) == e ? 1u << (4 * c + i) : 0;
            }
        } else {
            for (uint32_t i = 0; i < 16 && p0 + i < a.pairs; ++i) hits |= a.ids[p0 + i] == e ? 1u << i : 0;
        }
        uint32_t upto = __popc(hits);          // of the lanes up to this one
#pragma unroll
        for (int o = 1; o < 64; o *= 2) {
            const uint32_t w = __shfl_up(upto, o);
            upto += lane >= uint32_t(o) ? w : 0;
        }
        __syncthreads();                       // the last turn's sums have been read
        if (lane == 63) f.sums[wave] = upto;
        __syncthreads();
        uint32_t at = count + upto - __popc(hits);
#pragma unroll
        for (uint32_t o = 0; o < kTileThreads / 64; ++o) {
            at += o < wave ? f.sums[o] : 0;
            count += f.sums[o];
        }
        while (hits && at < kTileRows) {
            f.list[at++] = p0 + __builtin_ctz(hits);
            hits &= hits - 1;
        }
    }
    __syncthreads();
    return count < kTileRows ? count : kTileRows;
}

// UP: 64 rows of gate and of up; else 128 rows of down.
template <int WK, bool F16, Rows R, bool UP>
__global__ __launch_bounds__(kTileThreads, 2) void tile(Args a) {
    constexpr bool FP4 = is_fp4(WK), MX = is_mx(WK), GROUPED = WK == ST_KIND_FP8_BLOCK128;
    constexpr int PLANES = R == PLAIN ? 1 : 2, MT = kTileRows / 16, WC = FP4 ? 1 : 2;    // 16-byte chunks of a weight row per lane and step
    constexpr int PER = kTileRows * (kTileK / 8) / kTileThreads;                          // 16-byte chunks of x per thread, step and plane
    __shared__ __align__(16) uint8_t lds[2][PLANES][kTileRows * kTileK * 2];
    __shared__ Found found;
    const int tid = threadIdx.x, lane = tid & 63, row = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int32_t e = expert_of(a, blockIdx.y);
    if (e < 0) return;
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
    const uint32_t w_row = FP4 ? K / 2 : K, ws_row = K / (WK == ST_KIND_NVFP4 ? 16 : 32), groups = (K + 127) / 128, steps = (K + kTileK - 1) / kTileK;
    const uint64_t plane = uint64_t(a.pairs) * a.h_pitch * 2;

    for (uint32_t from = 0;;) {
        const uint32_t count = find(a, e, from, found);
        if (count == 0 || (a.by_pair && from == 0 && found.list[0] != blockIdx.y)) return;
        const int mt = int(count + 15) / 16;
        // chunk c of row r of a step sits at c ^ (r & 15)
        const uint8_t* src[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t r = (i * kTileThreads + tid) / 16, p = found.list[r < count ? r : 0];
            src[i] = UP ? a.x + uint64_t(p / a.top) * a.x_pitch * 2 : a.h + uint64_t(p) * a.h_pitch * 2;
        }
        const uint32_t c = tid % 16;
        u32x4 rx[PLANES][PER], rw[2][WC];
        uint32_t rs[2][WC];
        float rg[2];
        auto load = [&](uint32_t step) {
            const uint32_t k0 = step * kTileK;
            const bool whole = k0 + kTileK <= K;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int j = 0; j < WC; ++j) {
                    const uint32_t k = k0 + (FP4 ? 32 * q : 64 * j + 16 * q), to = FP4 ? k / 2 : k;
                    const uint8_t* p = mat[i].w + uint64_t(n[i]) * w_row + to;
                    rw[i][j] = whole ? u32x4(*reinterpret_cast<const u32x4_any*>(p)) : load_chunk(p, int64_t(w_row) - to);
                    if constexpr (WK == ST_KIND_NVFP4) {
                        const uint8_t* ps = mat[i].s + uint64_t(n[i]) * ws_row + k / 16;
                        rs[i][j] = whole ? *reinterpret_cast<const u16_any*>(ps) : load_codes(ps, int64_t(ws_row) - k / 16, 2);
                    } else if constexpr (MX) {
                        rs[i][j] = k < K ? mat[i].s[uint64_t(n[i]) * ws_row + k / 32] : 0;
                    }
                }
                if constexpr (GROUPED) rg[i] = reinterpret_cast<const float*>(mat[i].s)[uint64_t(n[i] / 128) * groups + step];
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if ((i * kTileThreads + tid) / 16 >= uint32_t(16 * mt)) continue;
                const uint8_t* p = src[i] + (uint64_t(k0) + 8 * c) * 2;
                const int64_t avail = (int64_t(K) - k0 - 8 * c) * 2;
                rx[0][i] = whole ? u32x4(*reinterpret_cast<const u32x4_any*>(p)) : load_chunk(p, avail);
                if constexpr (R == TWO) rx[1][i] = whole ? u32x4(*reinterpret_cast<const u32x4_any*>(p + plane)) : load_chunk(p + plane, avail);
            }
        };
        auto commit = [&](int buf) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint32_t r = (i * kTileThreads + tid) / 16;
                if (r >= uint32_t(16 * mt)) continue;
                if constexpr (R == SPLIT) split_f16(rx[0][i], rx[0][i], rx[1][i]);
#pragma unroll
                for (int p = 0; p < PLANES; ++p) *reinterpret_cast<u32x4*>(&lds[buf][p][(r * 16 + (c ^ (r & 15))) * 16]) = rx[p][i];
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
            // this step's weights to operands of four instructions, each 32 of K: lane group q's eight elements are chunk at(m) of x
            u32x4 wv[2][4];
            float gs[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                gs[i] = GROUPED ? rg[i] : 1.0f;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
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
                for (int m = 0; m < 4; ++m) {
                    const int at = FP4 ? 4 * q + m : 8 * (m / 2) + 2 * q + (m & 1);
#pragma unroll
                    for (int p = 0; p < PLANES; ++p) {
                        const u32x4 xv = *reinterpret_cast<const u32x4*>(&lds[buf][p][((16 * j + row) * 16 + (at ^ row)) * 16]);
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
            const uint32_t p = found.list[16 * j + row];
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
        if (count < kTileRows) return;
        from = found.list[kTileRows - 1] + 1;
        __syncthreads();
    }
}

}  // namespace
}  // namespace st_moe_impl
