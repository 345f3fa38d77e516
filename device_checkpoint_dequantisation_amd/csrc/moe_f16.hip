// st_moe's gate and up products for fp16 rows.
#include "moe_kernels.h"

namespace st_moe_impl {
namespace {

template <int WK>
void launch(const Args& a, bool few, hipStream_t s) {
    using D = Dense<ST_X_F16, WK>;
    if (few) {
        const uint32_t turns = (a.k + Few<ST_X_BF16, WK>::SS - 1) / Few<ST_X_BF16, WK>::SS, most = up_waves(WK);
        const uint32_t waves = turns < 1 ? 1 : turns < most ? turns : most;
        hipLaunchKernelGGL((up_few<ST_X_F16, WK>), dim3((a.i + 15) / 16, a.slots), dim3(64 * waves), 0, s, a);
    } else {
        hipLaunchKernelGGL((tile<WK, D::F16, D::SPLIT ? SPLIT : PLAIN, true>), dim3((a.i + 63) / 64, a.slots), dim3(kTileThreads), 0, s, a);
    }
}

}  // namespace

void launch_up_f16(const Args& a, uint32_t kind, bool few, hipStream_t s) {
    switch (kind) {
        case ST_KIND_FP8_TENSOR: return launch<ST_KIND_FP8_TENSOR>(a, few, s);
        case ST_KIND_FP8_BLOCK128: return launch<ST_KIND_FP8_BLOCK128>(a, few, s);
        case ST_KIND_NVFP4: return launch<ST_KIND_NVFP4>(a, few, s);
        case ST_KIND_MXFP8: return launch<ST_KIND_MXFP8>(a, few, s);
        case ST_KIND_MXFP4: return launch<ST_KIND_MXFP4>(a, few, s);
    }
}

}  // namespace st_moe_impl
