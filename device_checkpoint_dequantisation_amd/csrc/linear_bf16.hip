// st_linear for bf16 rows.
#include "linear_kernels.h"

void st_linear_impl::launch_bf16(const Args& a, const Plan& p, uint32_t kind, hipStream_t s) {
    switch (kind) {
        case ST_KIND_FP8_TENSOR: return launch<ST_X_BF16, ST_KIND_FP8_TENSOR>(a, p, s);
        case ST_KIND_FP8_BLOCK128: return launch<ST_X_BF16, ST_KIND_FP8_BLOCK128>(a, p, s);
        case ST_KIND_NVFP4: return launch<ST_X_BF16, ST_KIND_NVFP4>(a, p, s);
        case ST_KIND_MXFP8: return launch<ST_X_BF16, ST_KIND_MXFP8>(a, p, s);
        case ST_KIND_MXFP4: return launch<ST_X_BF16, ST_KIND_MXFP4>(a, p, s);
    }
}
