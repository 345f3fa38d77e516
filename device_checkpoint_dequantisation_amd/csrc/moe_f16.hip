// st_moe's gate and up products for fp16 rows.
#include "moe_kernels.h"

void st_moe_impl::launch_up_f16(const Args& a, uint32_t kind, Cut cut, hipStream_t s) {
    switch (kind) {
        case ST_KIND_FP8_TENSOR: return launch_up<ST_X_F16, ST_KIND_FP8_TENSOR>(a, cut, s);
        case ST_KIND_FP8_BLOCK128: return launch_up<ST_X_F16, ST_KIND_FP8_BLOCK128>(a, cut, s);
        case ST_KIND_NVFP4: return launch_up<ST_X_F16, ST_KIND_NVFP4>(a, cut, s);
        case ST_KIND_MXFP8: return launch_up<ST_X_F16, ST_KIND_MXFP8>(a, cut, s);
        case ST_KIND_MXFP4: return launch_up<ST_X_F16, ST_KIND_MXFP4>(a, cut, s);
    }
}
