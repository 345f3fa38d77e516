// What the host side of st_linear (linear.cpp) hands to its kernels (linear_kernels.h).
#pragma once

#include <hip/hip_runtime.h>

#include "st_internal.h"

namespace st_linear_impl {

// x types: st_x_type.  Weight kinds: st_kind.
constexpr bool is_q(int x) { return x >= ST_X_FP8_ROW; }
constexpr bool is_fp4(int w) { return w == ST_KIND_NVFP4 || w == ST_KIND_MXFP4; }
constexpr bool is_mx(int w) { return w == ST_KIND_MXFP8 || w == ST_KIND_MXFP4; }

// linear_one: weight rows per wavefront.
constexpr int kOneRows = 4;

// linear_few: groups of 16 weight rows per wavefront, and wavefronts per workgroup.  Two groups halve x's traffic for
// more registers: fp4, whose turn takes twice the x, gains (16 rows through NVFP4 [5120, 25600] on MI355X: 41.8 us with two,
// 47 with one), the 8-bit kinds lose (block FP8 [4096, 4096], 2 rows: 8.0 against 6.6 us).
constexpr int few_groups(int w) { return is_fp4(w) ? 2 : 1; }
constexpr int few_waves(int w) { return is_fp4(w) ? 4 : 8; }

struct Args {
    const uint8_t *x, *xs, *w, *ws, *ws2, *bias, *res;
    uint8_t* out;
    float* part;                 // [splits][m][n] fp32 partial sums, or null
    uint64_t x_pitch, res_pitch, out_pitch;   // elements
    uint32_t m, n, k;
    uint32_t act, bias_type, res_type, out_type;
    uint32_t splits, steps;      // steps of K per split
    uint32_t tiles_m, tiles_n;
    uint32_t vec;                // four consecutive outputs may be stored (and residuals loaded) together
};

// How a product is cut into workgroups.
struct Plan {
    bool direct;                 // rows start and end on 16 bytes: global memory to LDS without a detour
    bool tail;                   // direct, with a partial last step of K or scale words off 4 bytes
    bool f8;                     // the f8f6f4 matrix instructions
    bool one;                    // linear_one
    bool few;                    // linear_few
    uint32_t waves;              // of a workgroup of linear_one and linear_few
    uint32_t bm, bn, splits, steps;
    uint64_t part_bytes;
};

// Enqueue the product for weight kind `kind`; one source file per group of x types (linear_bf16.hip,
// linear_f16.hip, linear_fp8.hip), which keeps each compilation short.
void launch_bf16(const Args& a, const Plan& p, uint32_t kind, hipStream_t s);
void launch_f16(const Args& a, const Plan& p, uint32_t kind, hipStream_t s);
void launch_fp8(const Args& a, const Plan& p, uint32_t kind, hipStream_t s);

}  // namespace st_linear_impl
