// st_moe's gate and up products for fp16 rows.
#include "moe_kernels.h"

namespace st_moe_impl {
namespace {

template <int WK>
void launch(const Args& a, Cut cut, hipStream_t s) {
    using D = Dense<ST_X_F16, WK>;
    const uint32_t chunks = (a.k + One<WK>::E - 1) / One<WK>::E, turns = (a.k + Turn<WK>::SS - 1) / Turn<WK>::SS;
    const dim3 few((a.i + 15) / 16, a.slots), block(64 * even(turns, kUpWaves));
    by_end<WK>(a.k, [&](auto end) {
        constexpr Ends END = decltype(end)::value;
        switch (cut) {
            case ONE:
                hipLaunchKernelGGL((up_one<ST_X_F16, WK>), dim3((a.i + kUpColumns - 1) / kUpColumns, a.slots), dim3(64 * even((chunks + 63) / 64, kOneMaxWaves)), 0, s, a);
                break;
            case FEW:
            case SOME: hipLaunchKernelGGL((up_few<ST_X_F16, WK, END>), few, block, 0, s, a); break;
            case MANY:
                hipLaunchKernelGGL((tile<WK, D::F16, D::SPLIT ? SPLIT : PLAIN, true, kUpK, END>), dim3((a.i + 63) / 64, a.slots), dim3(kTileThreads), 0, s, a);
                break;
        }
    });
}

}  // namespace

void launch_up_f16(const Args& a, uint32_t kind, Cut cut, hipStream_t s) {
    switch (kind) {
        case ST_KIND_FP8_TENSOR: return launch<ST_KIND_FP8_TENSOR>(a, cut, s);
        case ST_KIND_FP8_BLOCK128: return launch<ST_KIND_FP8_BLOCK128>(a, cut, s);
        case ST_KIND_NVFP4: return launch<ST_KIND_NVFP4>(a, cut, s);
        case ST_KIND_MXFP8: return launch<ST_KIND_MXFP8>(a, cut, s);
        case ST_KIND_MXFP4: return launch<ST_KIND_MXFP4>(a, cut, s);
    }
}

}  // namespace st_moe_impl
