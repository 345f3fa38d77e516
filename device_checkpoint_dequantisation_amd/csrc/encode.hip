// 8-bit activations and the norm ahead of them: st_encode and st_rms_norm.
//   encode    v = x or silu(gate) * x;  code = e4m3(v / s)
//   rms_norm  h = x + residual;  y = h / sqrt(mean(h^2) + eps) * weight, in the output type or encoded like v
// with s = amax / 448 per row or per 128 columns (fp32), or the power of two at or above it per 32 (E8M0).
//
// Arithmetic.  A code changes by a whole e4m3 step where v / s passes the middle between two codes, so which side of a middle
// the quotient lies on is decided exactly:
//  * encode without a gate: v, and so amax and s, are exact in fp32.  The fp32 quotient names the middle that is nearest, and the
//    sign of fma(-middle, s, v), which is exact, says on which side of it v / s lies.
//  * a gate or a norm: v, amax and the quotient are kept in fp64 (x + residual and the sum of squares too).  For MX, whose scale
//    is a power of two, v in fp32, good to 2^-21, decides unless it comes within 2^-20 of a middle or amax that near to a
//    power of two's edge; then the wavefront does its chunk again in fp64 (about one in 100).
// A fp64 quotient is rounded correctly: a middle has 5 bits, s 24 and v 53, so a quotient that is not a middle is not rounded to one.
// (A gate of 31 makes x * silu(gate) differ from x * gate by 2^-45 of itself: such values do lie that near to middles.)  A norm's own
// fp64 roundings come to a few 2^-53: its quotients within 2^-49 of a middle count as the middle.
//
// Without a gate, and to MXFP8, both are bound by memory: every input is read once and stays in registers (chunks of 8 elements per lane, 16-byte
// loads) while the row's sums and maxima are taken; groups of 128 and 32 columns are 16 and 4 lanes.  Measured on MI355X: norm of
// 8192 x 5120 bf16 with residual to MXFP8 68 us (4.3 TB/s), silu-gated 4096 x 25600 bf16 to MXFP8 100-104 us (5.1 TB/s; 143 with
// expf and an IEEE division, 217 in fp64 throughout), 777 x 12288 fp16 rows to one scale each 16 us (28.6 in fp64).
// Gates and norms to the other kinds wait for fp64 arithmetic: gated 4096 x 25600 to groups 220-231 us, to one scale per row 276;
// norm of 8192 x 5120 with residual to groups 83, to one scale per row 81.
#include <hip/hip_runtime.h>

#include "st_device.h"

namespace {

using namespace st_dev;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

static_assert(sizeof(st_encode_args) == 72 && sizeof(st_rms_norm_args) == 104, "the ctypes declarations have these sizes");

constexpr uint32_t kThreads = 256;
constexpr float kE4m3Max = 448.0f;

struct Args {
    const uint8_t *x, *b, *w;    // b: the residual or the gate, or null
    uint8_t *h, *out, *scale;
    uint64_t m, x_pitch, b_pitch;
    uint32_t d, w_type, out_type;
    double eps;
};

// ------------------------------------------------------------------------- elements

// Eight elements of type E as loaded.
template <uint32_t E>
struct Raw {
    u32x4 v[E == ST_OUT_F32 ? 2 : 1];
    __device__ __forceinline__ float at(int i) const {
        if constexpr (E == ST_OUT_F32) return as_f32(v[i >> 2][i & 3]);
        const uint32_t u = v[0][i >> 1];
        if constexpr (E == ST_OUT_BF16) return as_f32(i & 1 ? u & 0xFFFF0000u : u << 16);
        return float(__builtin_bit_cast(_Float16, uint16_t(i & 1 ? u >> 16 : u)));
    }
};
template <uint32_t E>
constexpr uint32_t kSize = E == ST_OUT_F32 ? 4 : 2;

// Elements [col, col + 8) of a row of d, zeros behind its end.  VEC: d is a multiple of 8 and the row 16-byte aligned.
template <uint32_t E, bool VEC>
__device__ __forceinline__ Raw<E> load8(const uint8_t* row, uint32_t col, uint32_t d) {
    Raw<E> r;
    const uint8_t* p = row + uint64_t(col) * kSize<E>;
    if constexpr (VEC) {
        r.v[0] = col < d ? *reinterpret_cast<const u32x4*>(p) : u32x4{0, 0, 0, 0};
        if constexpr (E == ST_OUT_F32) r.v[1] = col < d ? *reinterpret_cast<const u32x4*>(p + 16) : u32x4{0, 0, 0, 0};
    } else {
#pragma unroll
        for (int k = 0; k < int(sizeof(r.v) / 4); ++k) r.v[k >> 2][k & 3] = 0;
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
            if (col + i >= d) continue;
            if constexpr (E == ST_OUT_F32) r.v[i >> 2][i & 3] = reinterpret_cast<const uint32_t*>(p)[i];
            else r.v[0][i >> 1] |= uint32_t(reinterpret_cast<const uint16_t*>(p)[i]) << (16 * (i & 1));
        }
    }
    return r;
}

__device__ __forceinline__ bool finite(double v) { return __builtin_fabs(v) <= 1.7976931348623157e308; }
__device__ __forceinline__ double silu64(double g) { return g / (1.0 + exp(-g)); }
// The same to 5 * 2^-24 of itself: exp(-g) = 2^t (1 + r ln 2) with t + r = -g log2(e), t the rounded product and r the rest, and the
// hardware's 2^t and 1 / x (an ulp each).  For g from kSiluLeast up; below, 2^t passes fp32's range (1 / x becomes subnormal, then 0,
// with a result that may be finite or NaN) and the caller takes silu64.
constexpr float kSiluLeast = -87.0f;
__device__ __forceinline__ float silu32(float g) {
    const float t = g * -1.44269504f;                                  // the nearest fp32 to log2(e), and what it lacks
    const float r = __builtin_fmaf(g, -1.44269504f, -t) + g * -1.92596299e-8f;
    const float e = __builtin_amdgcn_exp2f(t);
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(e, r * 0.69314718f, e));
}

// ------------------------------------------------------------------------- scales and codes

// The scale of a group whose largest finite magnitude is amax, and its reciprocal.
template <uint32_t KIND>
struct Scale {
    uint32_t bits;    // fp32 bits, or the E8M0 code
    double inv;
    __device__ __forceinline__ double value() const { return KIND == ST_X_MXFP8 ? 1.0 / inv : double(as_f32(bits)); }
    __device__ __forceinline__ explicit Scale(double amax) {
        if constexpr (KIND == ST_X_MXFP8) {
            // 448 = 1.75 * 2^8: with amax = f * 2^e, f in [1, 2), the power is e - 8 up to f = 1.75 and e - 7 above
            const uint64_t u = __builtin_bit_cast(uint64_t, amax);
            int e = int(u >> 52) - 1023 - 8 + ((u & 0xFFFFFFFFFFFFFull) > 0xC000000000000ull ? 1 : 0);
            e = e < -127 ? -127 : e > 127 ? 127 : e;
            if (amax == 0.0) e = 0;
            bits = uint32_t(e + 127);
            inv = __builtin_bit_cast(double, uint64_t(1023 - e) << 52);
        } else {
            float s = float(amax / 448.0);
            s = s < 1.1754943508222875e-38f ? 1.1754943508222875e-38f : s > 3.4028234663852886e38f ? 3.4028234663852886e38f : s;
            if (amax == 0.0) s = 1.0f;
            bits = as_u32(s);
            inv = 1.0 / double(s);
        }
    }
};

// v / s as an fp32 number that rounds to e4m3 as v / s itself does: truncated, with the lowest bit set where
// anything was cut off (a second rounding, to fewer bits, then sees on which side of a middle the value lies).
// NORM: v may be off by a few 2^-53 of itself.
template <uint32_t KIND, bool NORM>
__device__ __forceinline__ float quotient(double v, const Scale<KIND>& s) {
    double t = v * s.inv;
    // the correctly rounded quotient (a power of two's product is exact)
    if constexpr (KIND != ST_X_MXFP8) t = __builtin_fma(__builtin_fma(-t, s.value(), v), s.inv, t);
    if constexpr (NORM) t = __builtin_bit_cast(double, (__builtin_bit_cast(uint64_t, t) + 0x8u) & ~uint64_t(0xF));
    const float f = float(t);
    const double back = double(f);
    uint32_t u = as_u32(f);
    u -= __builtin_fabs(back) > __builtin_fabs(t) ? 1u : 0u;
    u |= back != t ? 1u : 0u;
    const float c = __builtin_fminf(__builtin_fmaxf(as_f32(u), -kE4m3Max), kE4m3Max);
    return finite(v) ? c : __builtin_nanf("");
}

// e4m3 code of v / s for exact fp32 v >= 0 and s, with inv = 1 / s to a few ulp.  The codes' middles lie at the mantissa's fourth
// bit; below 2^-6 codes are 2^-9 apart, as in the binade above it, so the quotient is looked at with 2^-6 added.
__device__ __forceinline__ uint32_t code_exact(float v, float s, float inv) {
    const float q = __builtin_fminf(v * inv, kE4m3Max);
    const bool sub = q < 0.015625f;
    const float lift = sub ? 0.015625f : 0.0f;
    const uint32_t z = as_u32(q + lift);
    const float middle = as_f32((z & 0xFFF00000u) | 0x00080000u) - lift;
    const float r = __builtin_fmaf(-middle, s, v);
    const uint32_t c = (z >> 20) - (sub ? 968u : 960u);        // 2^-6 has code 8 and exponent field 121 = 968 / 8
    const uint32_t up = r > 0.0f || (r == 0.0f && (c & 1)) ? 1u : 0u;
    const uint32_t code = c + up;
    return code < 0x7Eu ? code : 0x7Eu;
}
// Eight codes of exact fp32 values.
__device__ __forceinline__ void codes_exact(const float* v, float s, float inv, uint32_t& lo, uint32_t& hi) {
    lo = hi = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float m = __builtin_fabsf(v[i]);
        const uint32_t c = (m <= 3.4028234663852886e38f ? code_exact(m, s, inv) : 0x7Fu) | (as_u32(v[i]) >> 24 & 0x80u);
        (i < 4 ? lo : hi) |= c << (8 * (i & 3));
    }
}
__device__ __forceinline__ float finite_abs(float v) {
    const float m = __builtin_fabsf(v);
    return m <= 3.4028234663852886e38f ? m : 0.0f;
}
template <int LANES>
__device__ __forceinline__ float max_over(float v) {
#pragma unroll
    for (int o = 1; o < LANES; o *= 2) v = __builtin_fmaxf(v, __shfl_xor(v, o));
    return v;
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}

template <int LANES>
__device__ __forceinline__ double max_over(double v) {
#pragma unroll
    for (int o = 1; o < LANES; o *= 2) v = __builtin_fmax(v, __shfl_xor(v, o));
    return v;
}
template <int LANES>
__device__ __forceinline__ double sum_over(double v) {
#pragma unroll
    for (int o = 1; o < LANES; o *= 2) v += __shfl_xor(v, o);
    return v;
}

// Codes of eight values to columns [col, col + 8) of a row of d.
template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* row, uint32_t col, uint32_t d, uint32_t lo, uint32_t hi) {
    if constexpr (VEC) {
        if (col < d) *reinterpret_cast<u32x2*>(row + col) = u32x2{lo, hi};
    } else {
        for (uint32_t i = 0; i < 8; ++i)
            if (col + i < d) row[col + i] = uint8_t((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
}

// A group's scale, by one lane of it.
template <uint32_t KIND>
__device__ __forceinline__ void store_scale(const Args& a, uint64_t row, uint32_t col, uint32_t bits) {
    if (threadIdx.x % (KIND == ST_X_MXFP8 ? 4 : 16) == 0 && col < a.d) {
        if constexpr (KIND == ST_X_MXFP8) a.scale[row * (a.d / 32) + col / 32] = uint8_t(bits);
        else reinterpret_cast<uint32_t*>(a.scale)[row * ((a.d + 127) / 128) + col / 128] = bits;
    }
}

// Eight exact fp32 values of a chunk whose group is a few neighbouring lanes (128 or 32 columns): amax, scale and codes.
template <uint32_t KIND, bool VEC>
__device__ __forceinline__ void encode_exact(const Args& a, uint64_t row, uint32_t col, const float* v) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = __builtin_fmaxf(amax, finite_abs(v[i]));
    const Scale<KIND> s(double(max_over<(KIND == ST_X_MXFP8 ? 4 : 16)>(amax)));
    uint32_t lo, hi;
    codes_exact(v, float(s.value()), float(s.inv), lo, hi);
    store_codes<VEC>(a.out + row * a.d, col, a.d, lo, hi);
    store_scale<KIND>(a, row, col, s.bits);
}

// The same for values known in fp64 (wide(v)), and to a few 2^-24 in fp32 (v) unless this lane is `odd`.
template <uint32_t KIND, bool VEC, bool NORM, class Wide>
__device__ __forceinline__ void encode_group(const Args& a, uint64_t row, uint32_t col, const float* v, bool odd, Wide wide) {
    constexpr int LANES = KIND == ST_X_MXFP8 ? 4 : 16;
    uint32_t lo, hi, bits;
    bool again = true;
    if constexpr (KIND == ST_X_MXFP8) {
        float amax = 0.0f;
        // odd: something that fp32 does not settle
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float m = __builtin_fabsf(v[i]);
            odd |= !(m <= 3.4028234663852886e38f);
            amax = __builtin_fmaxf(amax, m);
        }
        amax = max_over<4>(amax);
        // amax = f 2^e: its power of two changes at f = 1.75; tiny groups (and empty ones) are left to fp64
        odd |= ((as_u32(amax) + 16 - 0x600000u) & 0x7FFFFFu) < 32 || amax < 1e-30f;
        const Scale<KIND> s((double(amax)));
        const float inv = float(s.inv);
        bits = s.bits;
        // codes do not fall as values rise: where v a little lower and a little higher have the same code, v itself has it
        const float less = inv * (1.0f - 0x1p-20f), more = inv * (1.0f + 0x1p-20f);
        lo = pack4(v[0] * less, v[1] * less, v[2] * less, v[3] * less);
        hi = pack4(v[4] * less, v[5] * less, v[6] * less, v[7] * less);
        odd |= lo != pack4(v[0] * more, v[1] * more, v[2] * more, v[3] * more) ||
               hi != pack4(v[4] * more, v[5] * more, v[6] * more, v[7] * more);
        again = __any(odd);
    }
    if (again) {
        double w[8], amax = 0.0;
        wide(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = __builtin_fmax(amax, finite(w[i]) ? __builtin_fabs(w[i]) : 0.0);
        const Scale<KIND> s(max_over<LANES>(amax));
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = quotient<KIND, NORM>(w[i], s);
        lo = pack4(q[0], q[1], q[2], q[3]);
        hi = pack4(q[4], q[5], q[6], q[7]);
        bits = s.bits;
    }
    store_codes<VEC>(a.out + row * a.d, col, a.d, lo, hi);
    store_scale<KIND>(a, row, col, bits);
}

// ------------------------------------------------------------------------- kernels

// encode by groups of 128 or 32 columns: no row structure, a lane per chunk of 8.  grid: chunks of a row (whole groups of 16
// lanes, so that no group crosses rows) by rows.
template <uint32_t E, uint32_t KIND, bool VEC, bool GATE>
__global__ __launch_bounds__(kThreads) void encode_groups(Args a, uint32_t rows_at_once) {
    const uint32_t col = (blockIdx.x * kThreads + threadIdx.x) * 8;      // past the row: loads zeros, stores nothing
    for (uint64_t row = blockIdx.y; row < a.m; row += rows_at_once) {
        const Raw<E> x = load8<E, VEC>(a.x + row * a.x_pitch * kSize<E>, col, a.d);
        float v[8];
        if constexpr (GATE) {
            const Raw<E> g = load8<E, VEC>(a.b + row * a.b_pitch * kSize<E>, col, a.d);
            float least = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                least = __builtin_fminf(least, g.at(k));
                v[k] = silu32(g.at(k)) * x.at(k);
            }
            encode_group<KIND, VEC, false>(a, row, col, v, least < kSiluLeast, [&](double* w) {
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] = silu64(double(g.at(k))) * double(x.at(k));
            });
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = x.at(k);
            encode_exact<KIND, VEC>(a, row, col, v);
        }
    }
}

enum { kNorm = 0, kEncodeRow = 1 };

// One row per TPR lanes; CH chunks per lane kept in registers, or with CH == 0 any number, read again in each
// pass.  NORM: KIND 0 writes y, else its codes.  kEncodeRow: one scale per row.
// B: there is a residual or a gate.
template <int OP, uint32_t E, uint32_t KIND, bool VEC, int TPR, int CH, bool B>
__global__ __launch_bounds__(TPR < int(kThreads) ? kThreads : TPR) void rows(Args a) {
    __shared__ double shared[2][TPR < 64 ? 1 : TPR / 64];
    constexpr uint32_t PER = TPR < int(kThreads) ? kThreads / TPR : 1;      // rows of a workgroup
    const uint64_t row = uint64_t(blockIdx.x) * PER + threadIdx.x / TPR;
    const uint32_t t = threadIdx.x % TPR, d = a.d;
    const bool live = row < a.m;       // the last workgroup may hold fewer rows
    const uint32_t dd = live ? d : 0;  // a row that is not there is empty
    const uint8_t* px = a.x + (live ? row : 0) * a.x_pitch * kSize<E>;
    const uint8_t* pb = a.b + (live ? row : 0) * a.b_pitch * kSize<E>;
    constexpr int N = CH ? CH : 1;
    Raw<E> rx[N], rb[B ? N : 1];
    auto fetch = [&](int c, uint32_t col) {
        rx[c] = load8<E, VEC>(px, col, dd);
        if constexpr (B) rb[c] = load8<E, VEC>(pb, col, dd);
    };
    if constexpr (CH != 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) fetch(c, (c * TPR + t) * 8);
    }
    // f(c, col) over this lane's chunks.  In the re-reading form every lane of a wavefront makes the same number of turns, so that
    // its groups of lanes stay whole.
    auto each = [&](auto f) {
        if constexpr (CH != 0) {
#pragma unroll
            for (int c = 0; c < CH; ++c) f(c, uint32_t(c * TPR + t) * 8);
        } else {
            for (uint64_t col = uint64_t(t) * 8; col - uint64_t(t) * 8 < d; col += TPR * 8) {
                const uint32_t at = col < d ? uint32_t(col) : (d + 7) / 8 * 8;
                fetch(0, at);
                f(0, at);
            }
        }
    };
    auto reduce = [&](double v, int slot, auto op) {
        if constexpr (TPR > 64) {
            if (threadIdx.x % 64 == 0) shared[slot][threadIdx.x / 64] = v;
            __syncthreads();
            v = shared[slot][0];
#pragma unroll
            for (int i = 1; i < TPR / 64; ++i) v = op(v, shared[slot][i]);
        }
        return v;
    };
    // h = x + residual: rounded to fp32 (from there h_out's 16-bit types round as they would from the sum itself), and as it is
    auto h_of = [&](int c, int i) {
        if constexpr (B) return rx[c].at(i) + rb[c].at(i);
        else return rx[c].at(i);
    };
    auto h64 = [&](int c, int i) {
        if constexpr (B) return double(rx[c].at(i)) + double(rb[c].at(i));
        else return double(rx[c].at(i));
    };
    double inv = 0.0;
    if constexpr (OP == kNorm) {
        double ss = 0.0;
        each([&](int c, uint32_t) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const double h = h64(c, i);
                ss = __builtin_fma(h, h, ss);
            }
        });
        ss = reduce(sum_over<64>(ss), 0, [](double p, double q) { return p + q; });
        inv = 1.0 / sqrt(ss / double(d) + a.eps);
    }
    // the weight of columns [col, col + 8); its elements may have any type
    auto weight = [&](uint32_t col, float* w) {
        if (!a.w) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 1.0f;
        } else if (VEC) {
            if (col < dd) {
                load4_as_f32(a.w, a.w_type, col, w);
                load4_as_f32(a.w, a.w_type, col + 4, w + 4);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = 0.0f;
            }
        } else {
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) w[i] = col + i < dd ? load_as_f32(a.w, a.w_type, col + i) : 0.0f;
        }
    };
    // the eight values to encode
    auto values = [&](int c, uint32_t col, double* v) {
        if constexpr (OP == kNorm) {
            float w[8];
            weight(col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = h64(c, i) * inv * double(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = double(rx[c].at(i));
                if constexpr (B) v[i] *= silu64(double(rb[c].at(i)));
            }
        }
    };
    // h goes out in the last pass: it may replace x or the residual, which the re-reading form still needs before
    auto store_h = [&](int c, uint32_t col) {
        if constexpr (OP == kNorm) {
            if (!a.h || col >= dd) return;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = h_of(c, i);
            if constexpr (VEC) {
                store4(a.h, E, row * d + col, v);
                store4(a.h, E, row * d + col + 4, v + 4);
            } else {
                for (uint32_t i = 0; i < 8; ++i)
                    if (col + i < d) store_as(a.h, E, row * d + col + i, v[i]);
            }
        }
    };
    if constexpr (KIND == 0) {
        each([&](int c, uint32_t col) {
            float w[8], y[8];
            weight(col, w);
            // in fp64: the factor of a row of the smallest values may lie beyond fp32
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = float(h64(c, i) * inv * double(w[i]));
            store_h(c, col);
            if constexpr (VEC) {
                if (col < dd) {
                    store4(a.out, a.out_type, row * d + col, y);
                    store4(a.out, a.out_type, row * d + col + 4, y + 4);
                }
            } else {
                for (uint32_t i = 0; i < 8; ++i)
                    if (col + i < dd) store_as(a.out, a.out_type, row * d + col + i, y[i]);
            }
        });
    } else if constexpr (KIND == ST_X_FP8_ROW) {
        if constexpr (OP == kEncodeRow && !B) {
            float amax = 0.0f;
            each([&](int c, uint32_t) {
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = __builtin_fmaxf(amax, finite_abs(rx[c].at(i)));
            });
            const Scale<KIND> s(reduce(double(max_over<64>(amax)), 1, [](double p, double q) { return __builtin_fmax(p, q); }));
            if (t == 0 && live) reinterpret_cast<uint32_t*>(a.scale)[row] = s.bits;
            const float inv = float(s.inv);
            each([&](int c, uint32_t col) {
                float v[8];
                uint32_t lo, hi;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = rx[c].at(i);
                codes_exact(v, as_f32(s.bits), inv, lo, hi);
                store_codes<VEC>(a.out + row * d, col, dd, lo, hi);
            });
        } else {
        // up to four chunks of fp64 values stay in registers between the passes (8192 x 5120 with residual: 81 us, 99 computed twice)
        constexpr bool KEEP = CH != 0 && CH <= 4;
        double kept[KEEP ? CH : 1][8];
        double amax = 0.0;
        each([&](int c, uint32_t col) {
            double* v = kept[KEEP ? c : 0];
            values(c, col, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = __builtin_fmax(amax, finite(v[i]) ? __builtin_fabs(v[i]) : 0.0);
        });
        amax = reduce(max_over<64>(amax), 1, [](double p, double q) { return __builtin_fmax(p, q); });
        const Scale<KIND> s(amax);
        if (t == 0 && live) reinterpret_cast<uint32_t*>(a.scale)[row] = s.bits;
        each([&](int c, uint32_t col) {
            double* v = kept[KEEP ? c : 0];
            float q[8];
            if constexpr (!KEEP) values(c, col, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = quotient<KIND, OP == kNorm>(v[i], s);
            store_h(c, col);
            store_codes<VEC>(a.out + row * d, col, dd, pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
        });
        }
    } else {
        const float s = float(inv);
        each([&](int c, uint32_t col) {
            float w[8], v[8];
            weight(col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = h_of(c, i) * s * w[i];
            store_h(c, col);
            // lanes of a row that is not there take part in the reductions and store nothing
            encode_group<KIND, VEC, true>(a, row, live ? col : (d + 7) / 8 * 8, v, false, [&](double* y) {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = h64(c, i) * inv * double(w[i]);
            });
        });
    }
}

// ------------------------------------------------------------------------- launches

constexpr uint32_t kMostBlocks = 1u << 22;     // of up to 512 threads

template <int OP, uint32_t E, uint32_t KIND, bool B>
void launch_rows(const Args& a, bool vec, hipStream_t s) {
    const uint32_t chunks = (a.d + 7) / 8;
    auto go = [&](auto kernel, uint32_t threads, uint32_t per_block) {
        // A grid holds fewer than 2^32 threads: more rows are launched in parts.  (A second grid dimension costs each call 1%.)
        Args part = a;
        for (uint64_t done = 0, most = uint64_t(kMostBlocks) * per_block; done < a.m; done += most) {
            part.m = a.m - done < most ? a.m - done : most;
            hipLaunchKernelGGL(kernel, dim3(uint32_t((part.m + per_block - 1) / per_block)), dim3(threads), 0, s, part);
            part.x += most * a.x_pitch * kSize<E>;
            if (B) part.b += most * a.b_pitch * kSize<E>;
            if (a.h) part.h += most * a.d * kSize<E>;
            part.out += most * a.d * (KIND != 0 ? 1 : a.out_type == ST_OUT_F32 ? 4 : 2);
            if (KIND != 0) part.scale += most * (KIND == ST_X_FP8_ROW ? 4 : KIND == ST_X_MXFP8 ? a.d / 32 : uint64_t(a.d + 127) / 128 * 4);
        }
    };
    // rows that are not whole aligned chunks, or do not fit the registers, are read again in each pass
    if (!vec || chunks > 4096 || (E == ST_OUT_F32 && chunks > 2048)) go(rows<OP, E, KIND, false, 256, 0, B>, 256, 1);
    else if (chunks <= 64) go(rows<OP, E, KIND, true, 64, 1, B>, 256, 4);
    else if (chunks <= 256) go(rows<OP, E, KIND, true, 256, 1, B>, 256, 1);
    else if (chunks <= 512) go(rows<OP, E, KIND, true, 256, 2, B>, 256, 1);
    else if (chunks <= 768) go(rows<OP, E, KIND, true, 256, 3, B>, 256, 1);
    else if (chunks <= 1024) go(rows<OP, E, KIND, true, 256, 4, B>, 256, 1);
    else if (chunks <= 2048) go(rows<OP, E, KIND, true, 512, 4, B>, 512, 1);
    else if constexpr (E != ST_OUT_F32) go(rows<OP, E, KIND, true, 512, 8, B>, 512, 1);
}
template <int OP, uint32_t E, uint32_t KIND>
void launch_rows(const Args& a, bool vec, hipStream_t s) {
    a.b ? launch_rows<OP, E, KIND, true>(a, vec, s) : launch_rows<OP, E, KIND, false>(a, vec, s);
}

template <uint32_t E, uint32_t KIND>
void launch_groups(const Args& a, bool vec, hipStream_t s) {
    const uint32_t lanes = (a.d + 127) / 128 * 16, rows_at_once = a.m < 32768 ? uint32_t(a.m) : 32768;
    const dim3 grid((lanes + kThreads - 1) / kThreads, rows_at_once);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, a, rows_at_once); };
    if (a.b) vec ? go(encode_groups<E, KIND, true, true>) : go(encode_groups<E, KIND, false, true>);
    else vec ? go(encode_groups<E, KIND, true, false>) : go(encode_groups<E, KIND, false, false>);
}

template <uint32_t E>
void launch_norm(const Args& a, uint32_t kind, bool vec, hipStream_t s) {
    switch (kind) {
        case ST_X_FP8_ROW: return launch_rows<kNorm, E, ST_X_FP8_ROW>(a, vec, s);
        case ST_X_FP8_GROUP128: return launch_rows<kNorm, E, ST_X_FP8_GROUP128>(a, vec, s);
        case ST_X_MXFP8: return launch_rows<kNorm, E, ST_X_MXFP8>(a, vec, s);
        default: return launch_rows<kNorm, E, 0>(a, vec, s);
    }
}
template <uint32_t E>
void launch_encode(const Args& a, uint32_t kind, bool vec, hipStream_t s) {
    switch (kind) {
        case ST_X_FP8_ROW: return launch_rows<kEncodeRow, E, ST_X_FP8_ROW>(a, vec, s);
        case ST_X_FP8_GROUP128: return launch_groups<E, ST_X_FP8_GROUP128>(a, vec, s);
        default: return launch_groups<E, ST_X_MXFP8>(a, vec, s);
    }
}

uint32_t size_of(uint32_t type) { return type == ST_OUT_F32 ? 4 : 2; }
bool off(const void* p, uint64_t n) { return p && reinterpret_cast<uintptr_t>(p) % n != 0; }

// What both entry points ask of their rows.
st_status check_rows(const char* who, const void* x, const void* b, uint64_t m, uint64_t d, uint64_t x_pitch,
                     uint64_t b_pitch, uint32_t type, uint32_t kind) {
    if (type > ST_OUT_F32) return st_fail(ST_E_ARG, "%s: unknown element type %u", who, type);
    if (m >= (uint64_t(1) << 31) || d >= (uint64_t(1) << 31))
        return st_fail(ST_E_SHAPE, "%s: m %llu, d %llu: each must be below 2^31", who, (unsigned long long)m, (unsigned long long)d);
    if (kind == ST_X_MXFP8 && d % 32) return st_fail(ST_E_SHAPE, "%s: MX d %llu is not a multiple of 32", who, (unsigned long long)d);
    if (m == 0 || d == 0) return ST_OK;
    if (!x) return st_fail(ST_E_ARG, "%s: null x", who);
    if (m > 1 && ((x_pitch < d && x_pitch != 0) || (b && b_pitch < d && b_pitch != 0)))
        return st_fail(ST_E_SHAPE, "%s: a row pitch is shorter than its row", who);
    if (off(x, size_of(type)) || off(b, size_of(type))) return st_fail(ST_E_ARG, "%s: a pointer is not aligned to its element type", who);
    return ST_OK;
}

bool rows_aligned(const void* p, uint64_t m, uint64_t pitch, uint32_t type) {
    return !p || (!off(p, 16) && (m <= 1 || pitch * size_of(type) % 16 == 0));
}

st_status launched(const char* who) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? ST_OK : st_fail(ST_E_HIP, "%s: launch failed: %s", who, hipGetErrorString(e));
}

}  // namespace

extern "C" st_status st_encode(const st_encode_args* g, void* stream) {
    const char* who = "st_encode";
    if (!g) return st_fail(ST_E_ARG, "%s: null arguments", who);
    if (g->kind < ST_X_FP8_ROW || g->kind > ST_X_MXFP8) return st_fail(ST_E_ARG, "%s: unknown encoding %u", who, g->kind);
    const st_status r = check_rows(who, g->x, g->gate, g->m, g->d, g->x_pitch, g->gate_pitch, g->x_type, g->kind);
    if (r != ST_OK) return r;
    if (g->m == 0) return ST_OK;
    if (!g->scale && (g->d || g->kind == ST_X_FP8_ROW)) return st_fail(ST_E_ARG, "%s: null scale", who);
    if (g->d && !g->data) return st_fail(ST_E_ARG, "%s: null data", who);
    if (g->kind != ST_X_MXFP8 && off(g->scale, 4)) return st_fail(ST_E_ARG, "%s: scale is not 4-byte aligned", who);
    if (g->d == 0 && g->kind != ST_X_FP8_ROW) return ST_OK;
    Args a = {};
    a.x = static_cast<const uint8_t*>(g->x);
    a.b = static_cast<const uint8_t*>(g->gate);
    a.out = static_cast<uint8_t*>(g->data);
    a.scale = static_cast<uint8_t*>(g->scale);
    a.m = g->m; a.d = uint32_t(g->d); a.x_pitch = g->x_pitch; a.b_pitch = g->gate_pitch;
    const bool vec = g->d % 8 == 0 && rows_aligned(g->x, g->m, g->x_pitch, g->x_type) &&
                     rows_aligned(g->gate, g->m, g->gate_pitch, g->x_type) && !off(g->data, 8);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (g->x_type == ST_OUT_BF16) launch_encode<ST_OUT_BF16>(a, g->kind, vec, s);
    else if (g->x_type == ST_OUT_F16) launch_encode<ST_OUT_F16>(a, g->kind, vec, s);
    else launch_encode<ST_OUT_F32>(a, g->kind, vec, s);
    return launched(who);
}

extern "C" st_status st_rms_norm(const st_rms_norm_args* g, void* stream) {
    const char* who = "st_rms_norm";
    if (!g) return st_fail(ST_E_ARG, "%s: null arguments", who);
    if (g->kind && (g->kind < ST_X_FP8_ROW || g->kind > ST_X_MXFP8)) return st_fail(ST_E_ARG, "%s: unknown encoding %u", who, g->kind);
    if (g->weight_type > ST_OUT_F32 || g->out_type > ST_OUT_F32) return st_fail(ST_E_ARG, "%s: unknown weight or output type", who);
    if (!(g->eps >= 0.0)) return st_fail(ST_E_ARG, "%s: eps %g is negative", who, g->eps);
    const st_status r = check_rows(who, g->x, g->residual, g->m, g->d, g->x_pitch, g->residual_pitch, g->x_type, g->kind);
    if (r != ST_OK) return r;
    if (g->m == 0) return ST_OK;
    if (!g->out && g->d) return st_fail(ST_E_ARG, "%s: null out", who);
    if (!g->scale && g->kind && (g->d || g->kind == ST_X_FP8_ROW)) return st_fail(ST_E_ARG, "%s: null scale", who);
    if (off(g->weight, size_of(g->weight_type)) || off(g->h_out, size_of(g->x_type)) ||
        (!g->kind && off(g->out, size_of(g->out_type))))
        return st_fail(ST_E_ARG, "%s: a pointer is not aligned to its element type", who);
    if (g->kind && g->kind != ST_X_MXFP8 && off(g->scale, 4)) return st_fail(ST_E_ARG, "%s: scale is not 4-byte aligned", who);
    if (g->d == 0 && g->kind != ST_X_FP8_ROW) return ST_OK;
    Args a = {};
    a.x = static_cast<const uint8_t*>(g->x);
    a.b = static_cast<const uint8_t*>(g->residual);
    a.w = static_cast<const uint8_t*>(g->weight);
    a.h = static_cast<uint8_t*>(g->h_out);
    a.out = static_cast<uint8_t*>(g->out);
    a.scale = static_cast<uint8_t*>(g->scale);
    a.m = g->m; a.d = uint32_t(g->d); a.x_pitch = g->x_pitch; a.b_pitch = g->residual_pitch;
    a.w_type = g->weight_type; a.out_type = g->out_type; a.eps = g->eps;
    const bool vec = g->d % 8 == 0 && rows_aligned(g->x, g->m, g->x_pitch, g->x_type) &&
                     rows_aligned(g->residual, g->m, g->residual_pitch, g->x_type) && !off(g->weight, 16) &&
                     !off(g->h_out, 16) && !off(g->out, 16);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (g->x_type == ST_OUT_BF16) launch_norm<ST_OUT_BF16>(a, g->kind, vec, s);
    else if (g->x_type == ST_OUT_F16) launch_norm<ST_OUT_F16>(a, g->kind, vec, s);
    else launch_norm<ST_OUT_F32>(a, g->kind, vec, s);
    return launched(who);
}
