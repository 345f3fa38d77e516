// st_linear for e4m3 rows (each weight kind has one encoding of x that goes with it).
#include "linear_kernels.h"

void st_linear_impl::launch_fp8(const Args& a, const Plan& p, uint32_t kind, hipStream_t s) {
    switch (kind) {
        case ST_KIND_FP8_TENSOR: return launch<ST_X_FP8_ROW, ST_KIND_FP8_TENSOR>(a, p, s);
        case ST_KIND_FP8_BLOCK128: return launch<ST_X_FP8_GROUP128, ST_KIND_FP8_BLOCK128>(a, p, s);
        case ST_KIND_MXFP8: return launch<ST_X_MXFP8, ST_KIND_MXFP8>(a, p, s);
        case ST_KIND_MXFP4: return launch<ST_X_MXFP8, ST_KIND_MXFP4>(a, p, s);
    }
}
