// st_kv_append: new keys and values into pages of e4m3 codes with one power of two for a block of tokens and a head.
//   s = the smallest power of two >= amax / 448 over the block's new tokens, or the block's scale if that is larger
//   code = v / s rounded to nearest even;  codes that were there: code * s_old / s, rounded again where s grew
// Dividing by a power of two is exact, so each code is rounded once (a code that is rounded again changes only below 2^-6 s), and
// fp32 holds everything.
//
// A workgroup has one block of tokens of one head, keys or values: nobody else writes its codes or its scale.  It reads the new tokens
// once and keeps them in registers until their amax is known, up to 32 numbers a lane (64 tokens of 128); larger blocks are read again from
// cache.  Bound by the new tokens' bytes where there are many (6 prompts' chunks of up to 2048 tokens, 8 heads of 128, read and written 38 MB: 15.3 us,
// 2.5 TB/s, a wave of workgroups that read, wait for each other and write), by the latency of four dependent loads where there are few
// (48 sequences' one token: 6.4 us).  Keys are stored as they come; values are turned, a lane taking two columns' 16 tokens, so that 16 bytes are stored together.
#include <hip/hip_runtime.h>

#include "kv_cache.h"

namespace {

using namespace st_kv;

static_assert(sizeof(st_kv_append_args) == 168, "the ctypes declaration has this size");

constexpr uint32_t kThreads = 256;

struct Args {
    Seqs s;
    const uint8_t *x[2];          // keys, values
    uint8_t *codes[2], *scale[2];
    uint64_t pitch[2], head_pitch[2];
    uint32_t head_dim;
};

template <uint32_t E>
__device__ __forceinline__ float element(const uint8_t* p, uint64_t i) {
    return load_as_f32(p, E, i);
}
// Eight elements at p + i; VEC: p and i are multiples of four elements.
template <uint32_t E, bool VEC>
__device__ __forceinline__ void load8(const uint8_t* p, uint64_t i, float* v) {
    if constexpr (VEC) {
        load4_as_f32(p, E, i, v);
        load4_as_f32(p, E, i + 4, v + 4);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = element<E>(p, i + k);
    }
}
// Two elements at p + i; VEC: in one load.
template <uint32_t E, bool VEC>
__device__ __forceinline__ void load2(const uint8_t* p, uint64_t i, float* v) {
    if constexpr (VEC && E == ST_OUT_F32) {
        const dword2 w = *reinterpret_cast<const dword2*>(p + 4 * i);
        v[0] = as_f32(w.x), v[1] = as_f32(w.y);
    } else if constexpr (VEC) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p + 2 * i);
        const f16x2 h = __builtin_bit_cast(f16x2, w);
        v[0] = E == ST_OUT_BF16 ? as_f32(w << 16) : float(h.x);
        v[1] = E == ST_OUT_BF16 ? as_f32(w & 0xFFFF0000u) : float(h.y);
    } else {
        v[0] = element<E>(p, i), v[1] = element<E>(p, i + 1);
    }
}
__device__ __forceinline__ bool finite(float v) { return __builtin_fabsf(v) <= 3.4028234663852886e38f; }

// a * 2^-e and b * 2^-e to codes in the low two bytes
__device__ __forceinline__ uint32_t codes2(float a, float b, int e) {
    const uint32_t c = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(__builtin_amdgcn_ldexpf(a, -e), __builtin_amdgcn_ldexpf(b, -e), 0, false)) & 0xFFFF;
    return (finite(a) ? c & 0xFF : 0x7F) | (finite(b) ? c & 0xFF00 : 0x7F00);
}
// four codes to the codes of their values * 2^-e
__device__ __forceinline__ uint32_t again4(uint32_t c, int e) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
    return codes2(lo.x, lo.y, e) | codes2(hi.x, hi.y, e) << 16;
}

template <uint32_t E, bool VEC>
__global__ __launch_bounds__(kThreads) void append(Args a) {
    __shared__ float most[kThreads / 64];
    const uint32_t head = blockIdx.x % a.s.heads, seq = blockIdx.y, which = blockIdx.z;
    const Span p = span_of(a.s, seq);
    const int64_t begin = p.pos < 0 ? 0 : p.pos, end = int64_t(p.pos) + p.count;
    const uint32_t block = 1u << a.s.block_log2, D = a.head_dim;
    const int64_t b = (begin >> a.s.block_log2) + blockIdx.x / a.s.heads, base = b << a.s.block_log2;
    if (base >= end) return;
    const int32_t page = page_of(a.s, seq, b);
    if (page < 0) return;
    const uint32_t lo = uint32_t(begin > base ? begin - base : 0), hi = uint32_t(end - base < block ? end - base : block);
    if (lo >= hi) return;
    const uint64_t at = uint64_t(page) * a.s.heads + head;
    const uint8_t* x = a.x[which];
    const uint64_t pitch = a.pitch[which];
    // element 0 of block token lo
    const uint64_t row0 = (uint64_t(p.first) + uint64_t(base + lo - p.pos)) * pitch + uint64_t(head) * a.head_pitch[which];
    uint8_t* codes = a.codes[which] + at * block * D;

    const uint32_t n = hi - lo, chunks = D / 8, items = n * chunks;       // keys: eight numbers of a token
    const uint32_t first = lo / 16, groups = (hi + 15) / 16 - first, pairs = D / 2, turned = groups * pairs;   // values: two columns of 16 tokens
    constexpr uint32_t KEEP = 4;
    const bool once = which == 0 ? items <= KEEP * kThreads : turned <= kThreads;
    float v[32];
    auto key = [&](uint32_t i, float* to) { load8<E, VEC>(x, row0 + uint64_t(i / chunks) * pitch + i % chunks * 8, to); };
    // value 2 t + c of item i: token t of its 16, column c of its two; 0 for tokens that are not new
    auto value = [&](uint32_t i, float* to) {
        const uint32_t d = i % pairs * 2, t0 = (first + i / pairs) * 16;
#pragma unroll
        for (uint32_t t = 0; t < 16; ++t) {
            const bool in = t0 + t >= lo && t0 + t < hi;
            const uint64_t o = row0 + uint64_t(in ? t0 + t - lo : 0) * pitch + d;
            load2<E, VEC>(x, o, to + 2 * t);
            to[2 * t] = in ? to[2 * t] : 0.0f;
            to[2 * t + 1] = in ? to[2 * t + 1] : 0.0f;
        }
    };
    float amax = 0.0f;
    auto more = [&](const float* from, int count) {
#pragma unroll
        for (int k = 0; k < count; ++k) amax = finite(from[k]) ? fmaxf(amax, __builtin_fabsf(from[k])) : amax;
    };
    if (once && which == 0) {
#pragma unroll
        for (uint32_t j = 0; j < KEEP; ++j) {
            const uint32_t i = threadIdx.x + j * kThreads;
            if (i < items) key(i, v + 8 * j);
            else
#pragma unroll
                for (int k = 0; k < 8; ++k) v[8 * j + k] = 0.0f;
        }
        more(v, 32);
    } else if (once) {
        if (threadIdx.x < turned) {
            value(threadIdx.x, v);
            more(v, 32);
        }
    } else {
        for (uint32_t i = threadIdx.x; i < items; i += kThreads) {
            key(i, v);
            more(v, 8);
        }
    }
#pragma unroll
    for (int o = 32; o; o /= 2) amax = fmaxf(amax, __shfl_xor(amax, o));
    if (threadIdx.x % 64 == 0) most[threadIdx.x / 64] = amax;
    // every thread has read the block's scale before thread 0 writes it below
    const int had = lo ? int(a.scale[which][at]) - 127 : -127;
    __syncthreads();
    amax = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
    // 448 = 1.75 * 2^8: with amax = f * 2^e, f in [1, 2), the power is e - 8 up to f = 1.75 and e - 7 above
    const uint32_t u = as_u32(amax);
    int e = int(u >> 23) - 127 - 8 + ((u & 0x7FFFFF) > 0x600000 ? 1 : 0);
    e = e < had ? had : e;
    const int up = e - had;       // >= 0

    if (which == 0) {
        auto put = [&](uint32_t i, const float* from) {
            *reinterpret_cast<dword2*>(codes + uint64_t(lo) * D + i * 8) =
                dword2{codes2(from[0], from[1], e) | codes2(from[2], from[3], e) << 16, codes2(from[4], from[5], e) | codes2(from[6], from[7], e) << 16};
        };
        if (once) {
#pragma unroll
            for (uint32_t j = 0; j < KEEP; ++j)
                if (threadIdx.x + j * kThreads < items) put(threadIdx.x + j * kThreads, v + 8 * j);
        } else {
            for (uint32_t i = threadIdx.x; i < items; i += kThreads) {
                key(i, v);
                put(i, v);
            }
        }
        if (up)
            for (uint32_t i = threadIdx.x; i < lo * chunks; i += kThreads) {
                dword2* c = reinterpret_cast<dword2*>(codes) + i;
                *c = dword2{again4(c->x, up), again4(c->y, up)};
            }
    } else {
        // 16 tokens of a column: those before lo are there already, those from hi on stay
        auto put = [&](uint32_t i, const float* from) {
            const uint32_t d = i % pairs * 2, t0 = (first + i / pairs) * 16;
#pragma unroll
            for (uint32_t col = 0; col < 2; ++col) {
                dword4* c = reinterpret_cast<dword4*>(codes + uint64_t(d + col) * block + t0);
                const bool all = t0 >= lo && t0 + 16 <= hi;
                const dword4 was = all ? dword4{0, 0, 0, 0} : *c;
                dword4 now;
#pragma unroll
                for (uint32_t w = 0; w < 4; ++w) {
                    uint32_t fresh = 0, old = 0;
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k) {
                        const uint32_t t = t0 + 4 * w + k;
                        fresh |= t >= lo && t < hi ? 0xFFu << 8 * k : 0;
                        old |= t < lo ? 0xFFu << 8 * k : 0;
                    }
                    const float* f = from + 8 * w + col;
                    const uint32_t code = codes2(f[0], f[2], e) | codes2(f[4], f[6], e) << 16;
                    const uint32_t kept = up && t0 < lo ? (again4(was[w], up) & old) | (was[w] & ~old) : was[w];
                    now[w] = (code & fresh) | (kept & ~fresh);
                }
                *c = now;
            }
        };
        if (once) {
            if (threadIdx.x < turned) put(threadIdx.x, v);
        } else {
            for (uint32_t i = threadIdx.x; i < turned; i += kThreads) {
                value(i, v);
                put(i, v);
            }
        }
        // whole groups of 16 tokens that were there before
        if (up)
            for (uint32_t i = threadIdx.x; i < first * D; i += kThreads) {
                dword4* c = reinterpret_cast<dword4*>(codes + uint64_t(i % D) * block + i / D * 16);
                const dword4 was = *c;
                *c = dword4{again4(was[0], up), again4(was[1], up), again4(was[2], up), again4(was[3], up)};
            }
    }
    if (threadIdx.x == 0) a.scale[which][at] = uint8_t(e + 127);
}

const char* kWho = "st_kv_append";

bool off(const void* p, uint64_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

}  // namespace

extern "C" st_status st_kv_append(const st_kv_append_args* g, void* stream) {
    if (!g) return st_fail(ST_E_ARG, "%s: null arguments", kWho);
    if (g->x_type > ST_OUT_F32) return st_fail(ST_E_ARG, "%s: unknown element type %u", kWho, g->x_type);
    if (g->head_dim == 0 || g->head_dim > 256 || g->head_dim % 32)
        return st_fail(ST_E_SHAPE, "%s: head_dim %u is not a multiple of 32 up to 256", kWho, g->head_dim);
    if (g->block != 16 && g->block != 32 && g->block != 64 && g->block != 128)
        return st_fail(ST_E_SHAPE, "%s: block %u is not 16, 32, 64 or 128", kWho, g->block);
    const uint64_t lim = uint64_t(1) << 31;
    if (g->tokens >= lim || g->max_new >= lim || g->pages >= lim || g->table_blocks >= lim / 2 / g->block || g->seqs > 65535 || g->heads > 65535)
        return st_fail(ST_E_SHAPE, "%s: %llu tokens, %llu sequences, %u heads, %llu pages or %llu blocks a sequence are too many", kWho,
                       (unsigned long long)g->tokens, (unsigned long long)g->seqs, g->heads, (unsigned long long)g->pages,
                       (unsigned long long)g->table_blocks);
    if (g->tokens == 0 || g->seqs == 0 || g->heads == 0 || g->pages == 0 || g->table_blocks == 0 || g->max_new == 0) return ST_OK;
    if (!g->starts && g->tokens % g->seqs)
        return st_fail(ST_E_SHAPE, "%s: %llu tokens are not %llu equal parts", kWho, (unsigned long long)g->tokens, (unsigned long long)g->seqs);
    if (!g->k_new || !g->v_new || !g->k || !g->v || !g->k_scale || !g->v_scale || !g->table || !g->lengths)
        return st_fail(ST_E_ARG, "%s: null pointer", kWho);
    if (g->seqs > 1 && g->table_pitch < g->table_blocks) return st_fail(ST_E_SHAPE, "%s: the table's pitch is shorter than its row", kWho);
    const uint64_t size = g->x_type == ST_OUT_F32 ? 4 : 2;
    if (off(g->k_new, size) || off(g->v_new, size)) return st_fail(ST_E_ARG, "%s: a pointer is not aligned to its element type", kWho);
    if (off(g->k, 16) || off(g->v, 16)) return st_fail(ST_E_ARG, "%s: the cache is not 16-byte aligned", kWho);
    if (off(g->table, 4) || off(g->lengths, 4) || off(g->starts, 4)) return st_fail(ST_E_ARG, "%s: a table is not 4-byte aligned", kWho);
    Args a = {};
    a.s = Seqs{g->table, g->lengths, g->starts, g->pages, g->table_blocks, g->table_pitch, uint32_t(g->tokens), uint32_t(g->seqs),
               uint32_t(g->max_new < g->tokens ? g->max_new : g->tokens), g->heads, stk::ilog2(g->block)};
    a.x[0] = static_cast<const uint8_t*>(g->k_new); a.x[1] = static_cast<const uint8_t*>(g->v_new);
    a.codes[0] = static_cast<uint8_t*>(g->k); a.codes[1] = static_cast<uint8_t*>(g->v);
    a.scale[0] = static_cast<uint8_t*>(g->k_scale); a.scale[1] = static_cast<uint8_t*>(g->v_scale);
    a.pitch[0] = g->k_pitch; a.pitch[1] = g->v_pitch; a.head_pitch[0] = g->k_head_pitch; a.head_pitch[1] = g->v_head_pitch;
    a.head_dim = g->head_dim;
    // blocks that new tokens of one sequence can touch
    const uint64_t per = g->starts ? a.s.max_new : g->tokens / g->seqs, count = per < a.s.max_new ? per : a.s.max_new;
    if (count == 0) return ST_OK;
    const uint64_t blocks = (count + g->block - 2) / g->block + 1;
    if (blocks * g->heads >= uint64_t(1) << 24) return st_fail(ST_E_SHAPE, "%s: %llu new tokens of %u heads are too many for one launch", kWho,
                                                               (unsigned long long)count, g->heads);
    const uint64_t v8 = 4 * size;     // load4_as_f32's alignment
    const bool vec = !off(g->k_new, v8) && !off(g->v_new, v8) && g->k_pitch % 4 == 0 && g->v_pitch % 4 == 0 &&
                     g->k_head_pitch % 4 == 0 && g->v_head_pitch % 4 == 0;
    const dim3 grid(uint32_t(blocks * g->heads), uint32_t(g->seqs), 2);
    hipStream_t s = static_cast<hipStream_t>(stream);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, a); };
    if (g->x_type == ST_OUT_BF16) vec ? go(append<ST_OUT_BF16, true>) : go(append<ST_OUT_BF16, false>);
    else if (g->x_type == ST_OUT_F16) vec ? go(append<ST_OUT_F16, true>) : go(append<ST_OUT_F16, false>);
    else vec ? go(append<ST_OUT_F32, true>) : go(append<ST_OUT_F32, false>);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? ST_OK : st_fail(ST_E_HIP, "%s: launch failed: %s", kWho, hipGetErrorString(e));
}
