// st_moe's down products and the sum over a token's experts.
#include "moe_kernels.h"

namespace st_moe_impl {
namespace {

// Pairs by expert: counted, placed and listed by one workgroup.  Which place a pair of an expert gets is left to the atomics' order, and
// changes no result: each pair's row is computed for itself.  5 us for 64 pairs and 5.5 for 2560: its barriers and a launch.
constexpr uint32_t kSortThreads = 1024;

__global__ __launch_bounds__(kSortThreads) void sort(Args a) {
    __shared__ uint32_t count[kMaxExperts];           // pairs of each expert, then where its next one goes
    __shared__ uint32_t sums[2][kSortThreads / 64];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (uint32_t e = tid; e < a.experts; e += kSortThreads) count[e] = 0;
    __syncthreads();
    for (uint32_t p = tid; p < a.pairs; p += kSortThreads) {
        const int32_t e = a.ids[p];
        if (e >= 0 && uint32_t(e) < a.experts) atomicAdd(&count[e], 1u);
    }
    uint32_t pairs = 0, entries = 0;                  // of the experts ahead
    for (uint32_t base = 0; base < a.experts; base += kSortThreads) {
        __syncthreads();
        const uint32_t e = base + tid, n = e < a.experts ? count[e] : 0, has = n ? 1 : 0;
        uint32_t upto = n;
#pragma unroll
        for (int o = 1; o < 64; o *= 2) {
            const uint32_t w = __shfl_up(upto, o);
            upto += lane >= uint32_t(o) ? w : 0;
        }
        const uint64_t m = __ballot(has);
        if (lane == 63) sums[0][wave] = upto, sums[1][wave] = __popcll(m);
        __syncthreads();
        uint32_t first = pairs + upto - n, at = entries + __popcll(m & ((uint64_t(1) << lane) - 1));
#pragma unroll
        for (uint32_t o = 0; o < kSortThreads / 64; ++o) {
            if (o < wave) first += sums[0][o], at += sums[1][o];
            pairs += sums[0][o], entries += sums[1][o];
        }
        if (has) *reinterpret_cast<u32x4*>(a.sorted + 4 + 4 * at) = u32x4{e, first, n, 0};
        if (e < a.experts) count[e] = first;
    }
    if (tid == 0) a.sorted[0] = entries;
    __syncthreads();
    for (uint32_t p = tid; p < a.pairs; p += kSortThreads) {
        const int32_t e = a.ids[p];
        if (e >= 0 && uint32_t(e) < a.experts) a.sorted[4 + 4 * a.slots + atomicAdd(&count[e], 1u)] = p;
    }
}

// A token's weighted results in the order of its experts: 320 tokens, 8 results of 4096 each (42 MB, mostly still in cache), 12 us.
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
void launch(const Args& a, Cut cut, hipStream_t s) {
    constexpr int NG = is_fp4(WK) ? 2 : 1;
    const dim3 grid((a.n + 16 * NG - 1) / (16 * NG)), block(64 * kDownWaves);
    by_end<WK>(a.i, [&](auto end) {
        constexpr Ends END = decltype(end)::value;
        switch (cut) {
            case ONE: {
                const uint64_t chunks = (uint64_t(a.i) + One<WK>::E - 1) / One<WK>::E * a.pairs;
                hipLaunchKernelGGL((down_one<WK>), dim3((a.n + kDownColumns - 1) / kDownColumns), dim3(64 * even((chunks + 63) / 64, kOneMaxWaves)), 0, s, a);
                break;
            }
            case FEW: hipLaunchKernelGGL((down_few<WK, NG, END>), grid, block, 0, s, a); break;
            case SOME:
            case MANY: {
                hipLaunchKernelGGL((tile<WK, false, TWO, false, down_k(WK), END>), dim3((a.n + 127) / 128, a.slots), dim3(kTileThreads), 0, s, a);
                const uint64_t items = uint64_t((a.n + 3) / 4) * a.t;
                hipLaunchKernelGGL(combine, dim3(uint32_t((items + 255) / 256)), dim3(256), 0, s, a);
            }
        }
    });
}

}  // namespace

void launch_sort(const Args& a, hipStream_t s) { hipLaunchKernelGGL(sort, dim3(1), dim3(kSortThreads), 0, s, a); }

void launch_down(const Args& a, uint32_t kind, Cut cut, hipStream_t s) {
    switch (kind) {
        case ST_KIND_FP8_TENSOR: return launch<ST_KIND_FP8_TENSOR>(a, cut, s);
        case ST_KIND_FP8_BLOCK128: return launch<ST_KIND_FP8_BLOCK128>(a, cut, s);
        case ST_KIND_NVFP4: return launch<ST_KIND_NVFP4>(a, cut, s);
        case ST_KIND_MXFP8: return launch<ST_KIND_MXFP8>(a, cut, s);
        case ST_KIND_MXFP4: return launch<ST_KIND_MXFP4>(a, cut, s);
    }
}

}  // namespace st_moe_impl
