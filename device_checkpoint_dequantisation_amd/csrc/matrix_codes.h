// Weight and cache codes as operands of the matrix instructions: what the kernels that multiply by quantised data share
// (linear_kernels.h, moe_kernels.h, attention.hip).
#pragma once

#include "linear.h"
#include "st_device.h"

namespace st_dev {

using st_linear_impl::is_fp4;
using st_linear_impl::is_mx;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// global memory takes vector loads at any byte
typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef uint64_t u64_any __attribute__((aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint16_t u16_any __attribute__((aligned(1)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float activate(float v, uint32_t act) {
    switch (act) {
        case ST_ACT_RELU: return v != v ? v : fmaxf(v, 0.0f);
        case ST_ACT_SILU: return silu(v);
        // (1 + erf z) / 2 as erfc(-z) / 2: 1 + erf cancels for negative z (4% off at v = -5, 0 from -5.5 on)
        case ST_ACT_GELU: return 0.5f * v * erfcf(v * -0.70710678118654752f);
        // (1 + tanh u) / 2 is the logistic function of 2u
        case ST_ACT_GELU_TANH: {
            const float u = 1.5957691216057308f * v * (1.0f + 0.044715f * v * v);
            return v / (1.0f + expf(-u));
        }
        default: return v;
    }
}

// ------------------------------------------------------------------------- weight codes to matrix operands

// Eight codes to eight bf16 or fp16 values times 2^e (s = 2^e; NVFP4: times the e4m3 block scale's value s).
// Exact within bf16's range (linear_kernels.h says what lies beyond it).  lo and hi: the eight e4m3 codes; fp4: lo alone.
template <bool F16, int WK>
__device__ __forceinline__ u32x4 codes8(uint32_t lo, uint32_t hi, float s) {
    u32x4 r;
    if constexpr (!is_fp4(WK)) {
        if constexpr (F16) {
            r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, s, false));
            r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, s, true));
            r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, s, false));
            r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, s, true));
        } else {
            r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false));
            r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true));
            r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false));
            r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true));
        }
    } else if constexpr (WK == ST_KIND_MXFP4) {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(lo, s, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(lo, s, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(lo, s, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(lo, s, 3));
    } else if constexpr (F16) {
        // 2^-10 <= |e2m1 * scale| <= 2688 with at most 6 bits: exact in fp16
        const f16x2 b = {_Float16(s), _Float16(s)};
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(lo, 1.0f, 0) * b);
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(lo, 1.0f, 1) * b);
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(lo, 1.0f, 2) * b);
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(lo, 1.0f, 3) * b);
    } else {
        f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, 1.0f, 0);
        r[0] = cvt_bf16x2(p.x * s, p.y * s);
        p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, 1.0f, 1);
        r[1] = cvt_bf16x2(p.x * s, p.y * s);
        p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, 1.0f, 2);
        r[2] = cvt_bf16x2(p.x * s, p.y * s);
        p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, 1.0f, 3);
        r[3] = cvt_bf16x2(p.x * s, p.y * s);
    }
    return r;
}

// The fp32 a scale code stands for: e4m3 (NVFP4), or E8M0 as the conversions above take it (the exponent
// field c: 2^(c - 127), 0 read as 2^-127 and 255 as NaN, checked on the device for every code).
template <int WK>
__device__ __forceinline__ float scale_of(uint32_t code) {
    if constexpr (WK == ST_KIND_NVFP4) return __builtin_amdgcn_cvt_pk_f32_fp8(code, false)[0];
    else if constexpr (is_mx(WK)) return as_f32(code << 23);
    else return 1.0f;
}

// 16x16x32 product of eight values per lane of each side.
template <bool F16>
__device__ __forceinline__ f32x4 mfma32(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// fp16 pairs as two bf16 terms, x = hi + lo: hi has the upper 8 of x's 11 significant bits, lo the rest.
__device__ __forceinline__ void split_f16(u32x4 x, u32x4& hi, u32x4& lo) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f16x2 h = __builtin_bit_cast(f16x2, uint32_t(x[i]));
        const float a = float(h.x), b = float(h.y);
        const uint32_t t = cvt_bf16x2(a, b);
        hi[i] = t;
        // infinities and NaN stay whole in hi
        const float la = a - as_f32(t << 16), lb = b - as_f32(t & 0xFFFF0000u);
        lo[i] = cvt_bf16x2(la == la ? la : 0.0f, lb == lb ? lb : 0.0f);
    }
}

// ------------------------------------------------------------------------- loads of rows that start anywhere

// 16 bytes at p of which `avail` lie in the row, the others 0.
__device__ __forceinline__ u32x4 load_chunk(const uint8_t* p, int64_t avail) {
    if (avail >= 16) return *reinterpret_cast<const u32x4_any*>(p);
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < avail) v[i >> 2] |= uint32_t(p[i]) << (8 * (i & 3));
    return v;
}
// The first `want` of the scale codes at p of which `avail` lie in the row, the others 0.
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t avail, int want) {
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < want && i < avail) v |= uint32_t(p[i]) << (8 * i);
    return v;
}

}  // namespace st_dev
