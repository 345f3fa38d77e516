// st_moe's down products and the sum over a token's experts.
#include "moe_kernels.h"

namespace st_moe_impl {
namespace {

// A token's weighted results in the order of its experts.
__global__ __launch_bounds__(256) void combine(Args a) {
    const uint32_t quads = (a.n + 3) / 4;
    const uint64_t i = uint64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= uint64_t(quads) * a.t) return;
    const uint32_t t = uint32_t(i / quads), n = uint32_t(i % quads) * 4;
    f32x4 v = {0, 0, 0, 0};
    for (uint32_t j = 0; j < a.top; ++j) {
        const uint32_t p = t * a.top + j;
        const int32_t e = a.ids[p];
        if (e < 0 || uint32_t(e) >= a.experts) continue;
        const float* from = a.part + uint64_t(p) * a.n + n;
        if ((a.n & 3) == 0) v += *reinterpret_cast<const f32x4*>(from);
        else
            for (uint32_t r = 0; r < 4 && n + r < a.n; ++r) v[r] += from[r];
    }
    store_y(a, t, n, v);
}

template <int WK>
void launch(const Args& a, bool few, hipStream_t s) {
    constexpr int NG = is_fp4(WK) ? 2 : 1;
    if (few) {
        hipLaunchKernelGGL((down_few<WK, NG>), dim3((a.n + 16 * NG - 1) / (16 * NG)), dim3(64 * kDownWaves), 0, s, a);
        return;
    }
    hipLaunchKernelGGL((tile<WK, false, TWO, false>), dim3((a.n + 127) / 128, a.slots), dim3(kTileThreads), 0, s, a);
    const uint64_t items = uint64_t((a.n + 3) / 4) * a.t;
    hipLaunchKernelGGL(combine, dim3(uint32_t((items + 255) / 256)), dim3(256), 0, s, a);
}

}  // namespace

void launch_down(const Args& a, uint32_t kind, bool few, hipStream_t s) {
    switch (kind) {
        case ST_KIND_FP8_TENSOR: return launch<ST_KIND_FP8_TENSOR>(a, few, s);
        case ST_KIND_FP8_BLOCK128: return launch<ST_KIND_FP8_BLOCK128>(a, few, s);
        case ST_KIND_NVFP4: return launch<ST_KIND_NVFP4>(a, few, s);
        case ST_KIND_MXFP8: return launch<ST_KIND_MXFP8>(a, few, s);
        case ST_KIND_MXFP4: return launch<ST_KIND_MXFP4>(a, few, s);
    }
}

}  // namespace st_moe_impl
