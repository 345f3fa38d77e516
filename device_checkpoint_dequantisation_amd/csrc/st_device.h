// Device helpers shared by the kernels that compute on activations (linear_kernels.h, encode.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "st_internal.h"

namespace st_dev {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t dword2 __attribute__((ext_vector_type(2)));
typedef uint32_t dword4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float as_f32(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ uint32_t as_u32(float f) { return __builtin_bit_cast(uint32_t, f); }
// fp32 pairs to bf16 / fp16 pairs, round to nearest even; a at the lower address
__device__ __forceinline__ uint32_t cvt_bf16x2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ uint32_t cvt_f16x2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2));
}

// Element i of an array of type t (st_out_dtype) as fp32.
__device__ __forceinline__ float load_as_f32(const uint8_t* p, uint32_t t, uint64_t i) {
    if (t == ST_OUT_BF16) return as_f32(uint32_t(reinterpret_cast<const uint16_t*>(p)[i]) << 16);
    if (t == ST_OUT_F16) return float(reinterpret_cast<const _Float16*>(p)[i]);
    return reinterpret_cast<const float*>(p)[i];
}
// Elements i..i+3, i a multiple of 4 and p aligned to four elements.
__device__ __forceinline__ void load4_as_f32(const uint8_t* p, uint32_t t, uint64_t i, float* v) {
    if (t == ST_OUT_F32) {
        const dword4 w = *reinterpret_cast<const dword4*>(p + 4 * i);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = as_f32(w[k]);
        return;
    }
    const dword2 w = *reinterpret_cast<const dword2*>(p + 2 * i);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (t == ST_OUT_BF16) {
            v[2 * k] = as_f32(w[k] << 16);
            v[2 * k + 1] = as_f32(w[k] & 0xFFFF0000u);
        } else {
            const f16x2 h = __builtin_bit_cast(f16x2, uint32_t(w[k]));
            v[2 * k] = float(h.x);
            v[2 * k + 1] = float(h.y);
        }
    }
}
__device__ __forceinline__ void store_as(uint8_t* p, uint32_t t, uint64_t i, float v) {
    if (t == ST_OUT_BF16) reinterpret_cast<uint16_t*>(p)[i] = uint16_t(cvt_bf16x2(v, 0.0f));
    else if (t == ST_OUT_F16) reinterpret_cast<_Float16*>(p)[i] = _Float16(v);
    else reinterpret_cast<float*>(p)[i] = v;
}
__device__ __forceinline__ void store4(uint8_t* p, uint32_t t, uint64_t i, const float* v) {
    if (t == ST_OUT_F32) *reinterpret_cast<dword4*>(p + 4 * i) = dword4{as_u32(v[0]), as_u32(v[1]), as_u32(v[2]), as_u32(v[3])};
    else if (t == ST_OUT_BF16) *reinterpret_cast<dword2*>(p + 2 * i) = dword2{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
    else *reinterpret_cast<dword2*>(p + 2 * i) = dword2{cvt_f16x2(v[0], v[1]), cvt_f16x2(v[2], v[3])};
}

__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

}  // namespace st_dev
