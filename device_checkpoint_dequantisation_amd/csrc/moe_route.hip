// st_moe_route: the router's scores and the choice of experts.
//   z = x router^T;  s = softmax(z) or 1 / (1 + e^-z);  the `top` largest, their weights
//
// Which experts are chosen must not depend on the order of a sum, so z is summed in 64 bits (products of 16-bit numbers are exact, the
// sums good to 2^-50), and everything behind it too.
//  * logits: a wavefront takes EW experts and TW tokens, eight elements of K per lane at a time, and folds the lanes' sums.
//  * choose: a token's scores in LDS; an expert's place is the number of those ahead of it, counted by one lane each, so that nothing
//    waits for a chain of maxima.
#include <hip/hip_runtime.h>

#include "matrix_codes.h"

namespace {

using namespace st_dev;

static_assert(sizeof(st_moe_route_args) == 120, "the ctypes declaration has this size");

struct Args {
    const uint8_t *x, *router;
    const float* bias;
    float* weights;
    int32_t* ids;
    double* z;                // [t, experts]
    uint64_t x_pitch, router_pitch;
    double scaling;
    uint32_t t, k, experts, top, sigmoid, renormalize;
};

constexpr int kWaves = 4;

// Eight elements of type E at element i of a row as fp32, zeros from k on; the row may start at any element.
template <uint32_t E>
__device__ __forceinline__ void load8(const uint8_t* p, uint32_t i, uint32_t k, float* v) {
    constexpr uint32_t S = E == ST_OUT_F32 ? 4 : 2;
    if (i + 8 <= k) {
        const u32x4 a = *reinterpret_cast<const u32x4_any*>(p + uint64_t(i) * S);
        if constexpr (E == ST_OUT_F32) {
            const u32x4 b = *reinterpret_cast<const u32x4_any*>(p + uint64_t(i) * S + 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = as_f32(a[j]), v[4 + j] = as_f32(b[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (E == ST_OUT_BF16) {
                    v[2 * j] = as_f32(a[j] << 16), v[2 * j + 1] = as_f32(a[j] & 0xFFFF0000u);
                } else {
                    const f16x2 h = __builtin_bit_cast(f16x2, uint32_t(a[j]));
                    v[2 * j] = float(h.x), v[2 * j + 1] = float(h.y);
                }
            }
        }
    } else {
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) v[j] = i + j < k ? load_as_f32(p, E, i + j) : 0.0f;
    }
}

template <uint32_t XE, uint32_t RE, int EW, int TW>
__global__ __launch_bounds__(64 * kWaves) void logits(Args a) {
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t e0 = (blockIdx.x * kWaves + wave) * EW, t0 = blockIdx.y * TW;
    if (e0 >= a.experts) return;
    constexpr uint32_t XS = XE == ST_OUT_F32 ? 4 : 2, RS = RE == ST_OUT_F32 ? 4 : 2;
    // experts and tokens past the last are read as the last one; nothing of them is stored
    const uint8_t *pr[EW], *px[TW];
#pragma unroll
    for (int i = 0; i < EW; ++i) pr[i] = a.router + uint64_t(e0 + i < a.experts ? e0 + i : a.experts - 1) * a.router_pitch * RS;
#pragma unroll
    for (int j = 0; j < TW; ++j) px[j] = a.x + uint64_t(t0 + j < a.t ? t0 + j : a.t - 1) * a.x_pitch * XS;
    double acc[EW][TW];
#pragma unroll
    for (int i = 0; i < EW; ++i)
#pragma unroll
        for (int j = 0; j < TW; ++j) acc[i][j] = 0.0;
    for (uint32_t k = lane * 8; k < a.k; k += 512) {
        float r[EW][8];
#pragma unroll
        for (int i = 0; i < EW; ++i) load8<RE>(pr[i], k, a.k, r[i]);
#pragma unroll
        for (int j = 0; j < TW; ++j) {
            float x[8];
            load8<XE>(px[j], k, a.k, x);
#pragma unroll
            for (int i = 0; i < EW; ++i)
#pragma unroll
                for (int c = 0; c < 8; ++c) acc[i][j] = __builtin_fma(double(r[i][c]), double(x[c]), acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < EW; ++i)
#pragma unroll
        for (int j = 0; j < TW; ++j) {
            double v = acc[i][j];
#pragma unroll
            for (int o = 32; o; o /= 2) v += __shfl_xor(v, o);
            if (lane == 0 && e0 + i < a.experts && t0 + j < a.t) a.z[uint64_t(t0 + j) * a.experts + e0 + i] = v;
        }
}

__device__ __forceinline__ double over_workgroup(double v, bool sum, double* shared) {
#pragma unroll
    for (int o = 32; o; o /= 2) {
        const double w = __shfl_xor(v, o);
        v = sum ? v + w : fmax(v, w);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
    __syncthreads();
    v = shared[0];
    for (uint32_t i = 1; i < blockDim.x >> 6; ++i) v = sum ? v + shared[i] : fmax(v, shared[i]);
    return v;
}

__global__ __launch_bounds__(1024) void choose(Args a) {
    __shared__ double key[1024], got[1024], shared[16];
    const uint32_t e = threadIdx.x;
    const uint64_t t = blockIdx.x;
    const bool in = e < a.experts;
    const double none = -__builtin_inf();
    const double z = in ? a.z[t * a.experts + e] : none;
    double s, total = 1.0;
    if (a.sigmoid) {
        s = in ? 1.0 / (1.0 + exp(-z)) : 0.0;
    } else {
        const double most = over_workgroup(z, false, shared);
        s = in ? exp(z - most) : 0.0;
        total = over_workgroup(s, true, shared);
        s /= total;
    }
    double mine = a.bias && in ? s + double(a.bias[e]) : z;
    if (mine != mine) mine = none;
    key[e] = mine;
    __syncthreads();
    uint32_t place = 0;
    for (uint32_t j = 0; j < a.experts; ++j) {
        const double other = key[j];
        place += other > mine || (other == mine && j < e) ? 1 : 0;
    }
    if (in && place < a.top) {
        a.ids[t * a.top + place] = int32_t(e);
        got[place] = s;
    }
    __syncthreads();
    if (in && place < a.top) {
        double w = s;
        if (a.renormalize) {
            double sum = 0.0;
            for (uint32_t j = 0; j < a.top; ++j) sum += got[j];
            w /= sum;
        }
        a.weights[t * a.top + place] = float(w * a.scaling);
    }
}

const char* kWho = "st_moe_route";

bool off(const void* p, uint64_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }
uint32_t size_of(uint32_t type) { return type == ST_OUT_F32 ? 4 : 2; }

st_status check_args(const st_moe_route_args* g) {
    if (!g) return st_fail(ST_E_ARG, "%s: null arguments", kWho);
    if (g->x_type > ST_OUT_F32 || g->router_type > ST_OUT_F32) return st_fail(ST_E_ARG, "%s: unknown element type", kWho);
    if (g->score > ST_ROUTE_SIGMOID || g->renormalize > 1) return st_fail(ST_E_ARG, "%s: score %u, renormalize %u", kWho, g->score, g->renormalize);
    if (g->experts == 0 || g->experts > 1024 || g->top == 0 || g->top > g->experts)
        return st_fail(ST_E_SHAPE, "%s: %u of %u experts; 1 to all of at most 1024 are needed", kWho, g->top, g->experts);
    if (g->t >= uint64_t(1) << 17 || g->k >= uint64_t(1) << 31)
        return st_fail(ST_E_SHAPE, "%s: t %llu must be below 2^17, k %llu below 2^31", kWho, (unsigned long long)g->t, (unsigned long long)g->k);
    if (g->t == 0) return ST_OK;
    if (!g->weights || !g->ids || (g->k && (!g->x || !g->router))) return st_fail(ST_E_ARG, "%s: null pointer", kWho);
    if ((g->t > 1 && g->x_pitch < g->k && g->x_pitch != 0) || (g->experts > 1 && g->router_pitch < g->k))
        return st_fail(ST_E_SHAPE, "%s: a row pitch is shorter than its row", kWho);
    if (off(g->x, size_of(g->x_type)) || off(g->router, size_of(g->router_type)) || off(g->bias, 4) || off(g->weights, 4) || off(g->ids, 4))
        return st_fail(ST_E_ARG, "%s: a pointer is not aligned to its element type", kWho);
    return ST_OK;
}

template <uint32_t XE, uint32_t RE>
void launch(const Args& a, hipStream_t s) {
    auto go = [&](auto kernel, uint32_t ew, uint32_t tw) {
        const dim3 grid((a.experts + kWaves * ew - 1) / (kWaves * ew), (a.t + tw - 1) / tw);
        hipLaunchKernelGGL(kernel, grid, dim3(64 * kWaves), 0, s, a);
    };
    if (a.t == 1) go(logits<XE, RE, 1, 1>, 1, 1);
    else go(logits<XE, RE, 4, 4>, 4, 4);
}
template <uint32_t XE>
void launch_router(const Args& a, uint32_t type, hipStream_t s) {
    if (type == ST_OUT_BF16) launch<XE, ST_OUT_BF16>(a, s);
    else if (type == ST_OUT_F16) launch<XE, ST_OUT_F16>(a, s);
    else launch<XE, ST_OUT_F32>(a, s);
}

}  // namespace

extern "C" st_status st_moe_route_workspace_bytes(const st_moe_route_args* g, uint64_t* bytes) {
    if (!bytes) return st_fail(ST_E_ARG, "st_moe_route_workspace_bytes: null bytes");
    *bytes = 0;
    const st_status r = check_args(g);
    if (r == ST_OK) *bytes = g->t * g->experts * 8;
    return r;
}

extern "C" st_status st_moe_route(const st_moe_route_args* g, void* stream) {
    const st_status r = check_args(g);
    if (r != ST_OK || g->t == 0) return r;
    const uint64_t need = g->t * g->experts * 8;
    if (!g->workspace || g->workspace_bytes < need)
        return st_fail(ST_E_ARG, "%s: %llu bytes of workspace, %llu are needed", kWho,
                       (unsigned long long)(g->workspace ? g->workspace_bytes : 0), (unsigned long long)need);
    if (off(g->workspace, 16)) return st_fail(ST_E_ARG, "%s: workspace is not 16-byte aligned", kWho);
    Args a = {};
    a.x = static_cast<const uint8_t*>(g->x); a.router = static_cast<const uint8_t*>(g->router);
    a.bias = g->bias; a.weights = g->weights; a.ids = g->ids; a.z = static_cast<double*>(g->workspace);
    a.x_pitch = g->x_pitch; a.router_pitch = g->router_pitch; a.scaling = g->scaling;
    a.t = uint32_t(g->t); a.k = uint32_t(g->k); a.experts = g->experts; a.top = g->top;
    a.sigmoid = g->score == ST_ROUTE_SIGMOID; a.renormalize = g->renormalize;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (g->x_type == ST_OUT_BF16) launch_router<ST_OUT_BF16>(a, g->router_type, s);
    else if (g->x_type == ST_OUT_F16) launch_router<ST_OUT_F16>(a, g->router_type, s);
    else launch_router<ST_OUT_F32>(a, g->router_type, s);
    hipLaunchKernelGGL(choose, dim3(a.t), dim3((a.experts + 63) / 64 * 64), 0, s, a);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? ST_OK : st_fail(ST_E_HIP, "%s: launch failed: %s", kWho, hipGetErrorString(e));
}
