// Host side of st_moe: argument checks, the cut into workgroups, the launches.
#include "moe.h"

#include <cstring>

namespace {

using namespace st_moe_impl;
using st_linear_impl::is_mx;

static_assert(sizeof(st_moe_args) == 152 && sizeof(st_moe_weight) == 24, "the ctypes declarations have these sizes");

const char* kWho = "st_moe";

bool off(const void* p, uint64_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }
uint32_t size_of(uint32_t t) { return t == ST_OUT_F32 ? 4 : 2; }

st_status check_kind(uint32_t kind, uint64_t k, const char* what) {
    if (kind < ST_KIND_FP8_TENSOR || kind > ST_KIND_MXFP4) return st_fail(ST_E_ARG, "%s: %s kind %u is not a quantised kind", kWho, what, kind);
    if ((kind == ST_KIND_NVFP4 && k % 16) || (is_mx(int(kind)) && k % 32))
        return st_fail(ST_E_SHAPE, "%s: %s kind %u with rows of %llu", kWho, what, kind, (unsigned long long)k);
    return ST_OK;
}

bool empty(const st_moe_args& g) { return g.t == 0 || g.n == 0; }

st_status check_args(const st_moe_args* g) {
    if (!g) return st_fail(ST_E_ARG, "%s: null arguments", kWho);
    if (g->x_type > ST_X_F16) return st_fail(ST_E_ARG, "%s: x type %u is not bf16 or fp16", kWho, g->x_type);
    if (g->activation > ST_ACT_GELU_TANH) return st_fail(ST_E_ARG, "%s: unknown activation %u", kWho, g->activation);
    if (g->residual_type > ST_OUT_F32 || g->out_type > ST_OUT_F32) return st_fail(ST_E_ARG, "%s: unknown residual or output type", kWho);
    const uint64_t lim = uint64_t(1) << 31;
    if (g->k >= lim || g->i >= lim || g->n >= lim || g->experts > kMaxExperts || g->top > kMaxTop || g->t >= lim || g->t * g->top >= uint64_t(1) << 24)
        return st_fail(ST_E_SHAPE, "%s: t %llu, k %llu, i %llu, n %llu, %u of %u experts are too many", kWho, (unsigned long long)g->t,
                       (unsigned long long)g->k, (unsigned long long)g->i, (unsigned long long)g->n, g->top, g->experts);
    st_status r = check_kind(g->up_kind, g->k, "gate and up");
    if (r == ST_OK) r = check_kind(g->down_kind, g->i, "down");
    if (r != ST_OK || empty(*g)) return r;
    if (g->k == 0 || g->i == 0 || g->experts == 0 || g->top == 0)
        return st_fail(ST_E_SHAPE, "%s: k %llu, i %llu, %u of %u experts", kWho, (unsigned long long)g->k, (unsigned long long)g->i, g->top, g->experts);
    if (!g->x || !g->ids || !g->weights || !g->experts_dev || !g->out) return st_fail(ST_E_ARG, "%s: null pointer", kWho);
    if (g->t > 1 && ((g->x_pitch < g->k && g->x_pitch != 0) || g->out_pitch < g->n ||
                     (g->residual && g->residual_pitch < g->n && g->residual_pitch != 0)))
        return st_fail(ST_E_SHAPE, "%s: a row pitch is shorter than its row", kWho);
    if (off(g->x, 2) || off(g->ids, 4) || off(g->weights, 4) || off(g->experts_dev, 8) || off(g->out, size_of(g->out_type)) ||
        off(g->residual, size_of(g->residual_type)))
        return st_fail(ST_E_ARG, "%s: a pointer is not aligned to its element type", kWho);
    return ST_OK;
}

struct Plan {
    Cut cut;
    uint64_t h_pitch, h_bytes, part_bytes, sort_bytes;
    uint64_t total() const { return h_bytes + part_bytes + sort_bytes; }
};

st_status plan_of(const st_moe_args& g, Plan* p) {
    const uint64_t pairs = g.t * g.top;
    const uint64_t slots = pairs < g.experts ? pairs : g.experts;
    // FEW: its down products go through all experts one after the other in every workgroup.  All in us, FEW's and SOME's: 32 pairs of 8 experts
    // (MXFP4 [1280, 4096]) 35 and 38, 64 of 128 (block FP8) 130 and 141, 64 of 64 (NVFP4 [1280, 5120]) 123 and 131, 128 of these 191 and
    // 199, 175 and 158, 128 of 128 (MXFP4 [768, 2048]) 84 and 59.
    // SOME: up_few reads an expert's weights from cache again for every 16 of its pairs, with a workgroup for each 16 of its columns; tiles of 64 are
    // too few workgroups, or mostly empty.  SOME's and MANY's: block FP8, 128 experts, 4 pairs each 312 and 385, 8 each 440 and 430, 12 each 540
    // and 504; kinds with scales of short blocks, whose decoding costs more: NVFP4, 64 experts, 8 each 323 and 381, 16 each 473 and 500, 24 each
    // 626 and 597; MXFP8 [768, 2048], 64 experts, 16 each 186 and 226; MXFP4, 32 experts, 16 each 259 and 302.
    const uint64_t each = g.up_kind <= ST_KIND_FP8_BLOCK128 ? 6 : 16;
    p->cut = g.t == 1 ? ONE : g.t <= 16 && pairs <= kFewPairs ? FEW : pairs <= slots * each ? SOME : MANY;
    p->h_pitch = (g.i + 7) / 8 * 8;
    p->h_bytes = (pairs * p->h_pitch * 4 + 15) / 16 * 16;
    p->part_bytes = p->cut >= SOME ? pairs * g.n * 4 : 0;
    p->part_bytes = (p->part_bytes + 15) / 16 * 16;
    p->sort_bytes = p->cut == ONE ? 0 : (4 + 4 * slots + pairs) * 4;
    // threads of each launch; a grid dimension holds fewer than 2^32, and 65535 workgroups in y (slots is below that)
    if ((g.i + 1) / 2 * 512 >> 32 || (g.n + 1) / 2 * 512 >> 32 || (p->cut >= SOME && (g.n + 3) / 4 * g.t >> 32) || slots > 65535)
        return st_fail(ST_E_SHAPE, "%s: i %llu, n %llu, t %llu take more threads than one launch holds", kWho, (unsigned long long)g.i,
                       (unsigned long long)g.n, (unsigned long long)g.t);
    return ST_OK;
}

}  // namespace

extern "C" st_status st_moe_workspace_bytes(const st_moe_args* g, uint64_t* bytes) {
    if (!bytes) return st_fail(ST_E_ARG, "st_moe_workspace_bytes: null bytes");
    *bytes = 0;
    const st_status r = check_args(g);
    if (r != ST_OK || empty(*g)) return r;
    Plan p;
    const st_status f = plan_of(*g, &p);
    if (f == ST_OK) *bytes = p.total();
    return f;
}

extern "C" st_status st_moe(const st_moe_args* g, void* stream) {
    const st_status r = check_args(g);
    if (r != ST_OK || empty(*g)) return r;
    Plan p;
    const st_status f = plan_of(*g, &p);
    if (f != ST_OK) return f;
    const uint64_t need = p.total();
    if (!g->workspace || g->workspace_bytes < need)
        return st_fail(ST_E_ARG, "%s: %llu bytes of workspace, %llu are needed", kWho,
                       (unsigned long long)(g->workspace ? g->workspace_bytes : 0), (unsigned long long)need);
    if (off(g->workspace, 16)) return st_fail(ST_E_ARG, "%s: workspace is not 16-byte aligned", kWho);
    Args a;
    memset(&a, 0, sizeof a);
    a.x = static_cast<const uint8_t*>(g->x);
    a.ids = g->ids; a.weights = g->weights; a.experts_dev = g->experts_dev;
    a.res = static_cast<const uint8_t*>(g->residual);
    a.out = static_cast<uint8_t*>(g->out);
    a.h = static_cast<uint8_t*>(g->workspace);
    a.part = p.part_bytes ? reinterpret_cast<float*>(a.h + p.h_bytes) : nullptr;
    a.x_pitch = g->x_pitch; a.res_pitch = g->residual_pitch; a.out_pitch = g->out_pitch; a.h_pitch = p.h_pitch;
    a.t = uint32_t(g->t); a.k = uint32_t(g->k); a.i = uint32_t(g->i); a.n = uint32_t(g->n);
    a.experts = g->experts; a.top = g->top; a.pairs = uint32_t(g->t * g->top);
    a.slots = p.cut == ONE || a.pairs < a.experts ? a.pairs : a.experts;
    a.sorted = reinterpret_cast<uint32_t*>(a.h + p.h_bytes + p.part_bytes);
    a.act = g->activation; a.res_type = g->residual_type; a.out_type = g->out_type;
    auto quad = [](const void* v, uint32_t type, uint64_t pitch, uint64_t rows) {
        return !off(v, 4 * size_of(type)) && (rows <= 1 || pitch % 4 == 0);
    };
    a.vec = quad(g->out, g->out_type, g->out_pitch, g->t) && (!g->residual || quad(g->residual, g->residual_type, g->residual_pitch, g->t));
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (p.cut != ONE) launch_sort(a, s);
    (g->x_type == ST_X_F16 ? launch_up_f16 : launch_up_bf16)(a, g->up_kind, p.cut, s);
    launch_down(a, g->down_kind, p.cut, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return st_fail(ST_E_HIP, "%s: launch failed: %s", kWho, hipGetErrorString(e));
    return ST_OK;
}
