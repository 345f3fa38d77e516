// st_moe_route: the router's scores and the choice of experts.
//   z = x router^T;  s = softmax(z) or 1 / (1 + e^-z);  the `top` largest, their weights
//
// Which experts are chosen must not depend on the order of a sum, so z is summed in 64 bits (products of 16-bit numbers are exact, the
// sums good to 2^-50), and everything behind it too.
//  * logits: 16 tokens by 16 experts a workgroup, on the fp64 matrix instructions (16 x 16 x 4, 64 cycles), which take one converted number
//    per lane and side; the wavefronts have parts of K and join in LDS.  777 tokens, 256 experts of 5120: bound by those instructions
//    (2 GFLOP at the 68 TFLOP/s that a large fp64 product reaches: 30 us) and by how 784 tiles
//    go into 256 CUs: 60 us.
//  * choose: a token's scores in LDS; an expert's place is the number of those ahead of it, counted by one lane each, so that nothing
//    waits for a chain of maxima.  777 tokens, 256 experts: 10.5 us; one token, 128 experts: 4.8, of which the launch is most.
#include <hip/hip_runtime.h>

#include <type_traits>

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

constexpr int kMaxWaves = 16;
typedef double f64x4 __attribute__((ext_vector_type(4)));

// Eight elements of type E at element i of a row as fp32, zeros from k on; the row may start at any element.
template <uint32_t E, bool WHOLE>
__device__ __forceinline__ void load8(const uint8_t* p, uint32_t i, uint32_t k, float* v) {
    constexpr uint32_t S = E == ST_OUT_F32 ? 4 : 2;
    if (WHOLE || i + 8 <= k) {
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

template <uint32_t XE, uint32_t RE>
__global__ __launch_bounds__(64 * kMaxWaves) void logits(Args a) {
    __shared__ double joined[kMaxWaves][256];
    const uint32_t lane = threadIdx.x & 63, row = lane & 15, g = lane >> 4, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const uint32_t e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
    constexpr uint32_t XS = XE == ST_OUT_F32 ? 4 : 2, RS = RE == ST_OUT_F32 ? 4 : 2;
    // experts and tokens past the last are read as the last one; nothing of them is stored
    const uint8_t* pr = a.router + uint64_t(e0 + row < a.experts ? e0 + row : a.experts - 1) * a.router_pitch * RS;
    const uint8_t* px = a.x + uint64_t(t0 + row < a.t ? t0 + row : a.t - 1) * a.x_pitch * XS;
    f64x4 acc = {0, 0, 0, 0};
    // 32 of K a turn: lane group g has eight of them, instruction i takes the i-th of each
    auto turn = [&](uint32_t k, auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        float r[8], x[8];
        load8<RE, WHOLE>(pr, k + 8 * g, a.k, r);
        load8<XE, WHOLE>(px, k + 8 * g, a.k, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc = __builtin_amdgcn_mfma_f64_16x16x4f64(double(x[i]), double(r[i]), acc, 0, 0, 0);
    };
    const uint32_t whole = a.k / 32;
    uint32_t i = wave;
    // (four turns' loads together)
#pragma unroll 4
    for (; i < whole; i += waves) turn(i * 32, std::true_type{});
    if (i * 32 < a.k) turn(i * 32, std::false_type{});
#pragma unroll
    for (int i = 0; i < 4; ++i) joined[wave][i * 64 + lane] = acc[i];
    __syncthreads();
    for (uint32_t o = threadIdx.x; o < 256; o += blockDim.x) {
        double v = joined[0][o];
        for (uint32_t w = 1; w < waves; ++w) v += joined[w][o];
        // result i of lane (row, g): token 4 i + g, expert `row`
        const uint32_t t = t0 + 4 * (o >> 6) + (o >> 4 & 3), e = e0 + (o & 15);
        if (t < a.t && e < a.experts) a.z[uint64_t(t) * a.experts + e] = v;
    }
}

// One token: a wavefront an expert, dot products on the vector unit (128 experts of 4096: 6 us, 15 on the matrix instructions, which would
// leave 15 of 16 rows empty and give eight workgroups all the router).
constexpr int kOneWaves = 4;
template <uint32_t XE, uint32_t RE>
__global__ __launch_bounds__(64 * kOneWaves) void logits_one(Args a) {
    const uint32_t lane = threadIdx.x & 63, e = blockIdx.x * kOneWaves + (threadIdx.x >> 6);
    if (e >= a.experts) return;
    const uint8_t* pr = a.router + uint64_t(e) * a.router_pitch * (RE == ST_OUT_F32 ? 4 : 2);
    double acc = 0.0;
    auto turn = [&](uint32_t k, auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        float r[8], x[8];
        load8<RE, WHOLE>(pr, k, a.k, r);
        load8<XE, WHOLE>(a.x, k, a.k, x);
#pragma unroll
        for (int c = 0; c < 8; ++c) acc = __builtin_fma(double(r[c]), double(x[c]), acc);
    };
    uint32_t k = 0;
#pragma unroll 4
    for (; k + 512 <= a.k; k += 512) turn(k + lane * 8, std::true_type{});
    if (k + lane * 8 < a.k) turn(k + lane * 8, std::false_type{});
#pragma unroll
    for (int o = 32; o; o /= 2) acc += __shfl_xor(acc, o);
    if (lane == 0) a.z[e] = acc;
}

// The largest of the workgroup's values, NaN if there is one, or their sum; in one order.
template <bool SUM>
__device__ __forceinline__ double over_workgroup(double v, double* shared) {
    auto join = [](double p, double q) { return SUM ? p + q : q > p ? q : q != q ? q : p; };
#pragma unroll
    for (int o = 32; o; o /= 2) v = join(v, __shfl_xor(v, o));
    if (blockDim.x == 64) return v;
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
    __syncthreads();
    v = shared[0];
    for (uint32_t i = 1; i < blockDim.x >> 6; ++i) v = join(v, shared[i]);
    return v;
}

typedef double f64x2 __attribute__((ext_vector_type(2)));

__global__ __launch_bounds__(1024) void choose(Args a) {
    __shared__ __align__(16) double key[1024], got[1024], shared[2][16];
    const uint32_t e = threadIdx.x;
    const uint64_t t = blockIdx.x;
    const bool in = e < a.experts;
    const double none = -__builtin_inf();
    const double z = in ? a.z[t * a.experts + e] : none;
    double s;
    if (a.sigmoid) {
        s = in ? 1.0 / (1.0 + exp(-z)) : 0.0;
    } else {
        const double most = over_workgroup<false>(z, shared[0]);      // (all lanes take part)
        s = in ? exp(z - most) : 0.0;
        // (weights that are divided by their own sum need no other)
        if (a.bias || !a.renormalize) s /= over_workgroup<true>(s, shared[1]);
    }
    double mine = a.bias && in ? s + double(a.bias[e]) : z;
    if (mine != mine) mine = none;
    key[e] = in ? mine : none;
    __syncthreads();
    // those ahead: larger ones, and equal ones of a smaller number, which all of the wavefronts before this one's are and none behind it
    // (keys behind the last expert are the least and have the largest numbers)
    uint32_t place = 0;
    const uint32_t mine0 = e & ~63u;
#pragma unroll 4
    for (uint32_t j = 0; j < mine0; j += 2) {
        const f64x2 other = *reinterpret_cast<const f64x2*>(&key[j]);
        place += uint32_t(other.x >= mine) + uint32_t(other.y >= mine);
    }
#pragma unroll 4
    for (uint32_t j = mine0; j < mine0 + 64; j += 2) {
        const f64x2 other = *reinterpret_cast<const f64x2*>(&key[j]);
        place += uint32_t(other.x > mine) + (uint32_t(other.x == mine) & uint32_t(j < e));
        place += uint32_t(other.y > mine) + (uint32_t(other.y == mine) & uint32_t(j + 1 < e));
    }
#pragma unroll 4
    for (uint32_t j = mine0 + 64; j < blockDim.x; j += 2) {
        const f64x2 other = *reinterpret_cast<const f64x2*>(&key[j]);
        place += uint32_t(other.x > mine) + uint32_t(other.y > mine);
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
    if (a.t == 1) {
        hipLaunchKernelGGL((logits_one<XE, RE>), dim3((a.experts + kOneWaves - 1) / kOneWaves), dim3(64 * kOneWaves), 0, s, a);
        return;
    }
    // few tiles: more wavefronts for each
    const uint32_t tiles_e = (a.experts + 15) / 16, tiles_t = (a.t + 15) / 16, turns = (a.k + 31) / 32;
    const uint32_t most = uint64_t(tiles_e) * tiles_t < 256 ? kMaxWaves : 4, waves = turns < 1 ? 1 : turns < most ? turns : most;
    hipLaunchKernelGGL((logits<XE, RE>), dim3(tiles_e, tiles_t), dim3(64 * waves), 0, s, a);
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
