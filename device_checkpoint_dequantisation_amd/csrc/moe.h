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
    uint32_t* sorted;             // [4 + 4 * slots + pairs]: their number, the experts that have pairs ({expert, first, pairs, 0} each), pairs by expert
    uint32_t slots;               // experts that can have pairs
    uint32_t act, res_type, out_type;
    uint32_t vec;                 // four consecutive outputs may be stored (and residuals loaded) together
};

constexpr uint32_t kMaxTop = 32, kMaxExperts = 16384, kFewPairs = 64;

// How the work is cut (moe_kernels.h): for one token; up_few and down_few; up_few and tiles of down; tiles.
enum Cut { ONE, FEW, SOME, MANY };

// The fewest wavefronts, at most `most`, that go through n items in as many rounds as `most` would.
inline uint32_t even(uint64_t n, uint32_t most) {
    if (n == 0) return 1;
    const uint64_t rounds = (n + most - 1) / most;
    return uint32_t((n + rounds - 1) / rounds);
}

void launch_sort(const Args& a, hipStream_t s);
void launch_up_bf16(const Args& a, uint32_t kind, Cut cut, hipStream_t s);
void launch_up_f16(const Args& a, uint32_t kind, Cut cut, hipStream_t s);
void launch_down(const Args& a, uint32_t kind, Cut cut, hipStream_t s);

}  // namespace st_moe_impl
