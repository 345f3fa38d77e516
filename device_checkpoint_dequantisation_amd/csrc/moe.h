// What the host side of st_moe (moe.cpp) hands to its kernels (moe_kernels.h).
#pragma once

#include "linear.h"

namespace st_moe_impl {

struct Args {
    const uint8_t* x;
    const int32_t* ids;
    const float* weights;
    const st_moe_weight* experts_dev;
    const uint8_t* res;
    uint8_t* out;
    uint8_t* h;                   // [2][pairs][h_pitch] bf16: act(gate x) * (up x) as two terms
    float* part;                  // [pairs][n] fp32: the experts' weighted results, or null
    uint64_t x_pitch, res_pitch, out_pitch, h_pitch;   // elements
    uint32_t t, k, i, n, experts, top, pairs;
    uint32_t slots, by_pair;      // grid of experts: the pairs' ids (the first pair of each expert works), or all experts
    uint32_t act, res_type, out_type;
    uint32_t vec;                 // four consecutive outputs may be stored (and residuals loaded) together
};

constexpr uint32_t kFewTokens = 16, kMaxTop = 32;

void launch_up_bf16(const Args& a, uint32_t kind, bool few, hipStream_t s);
void launch_up_f16(const Args& a, uint32_t kind, bool few, hipStream_t s);
void launch_down(const Args& a, uint32_t kind, bool few, hipStream_t s);

}  // namespace st_moe_impl
