// st_kv_attention: attention over pages of e4m3 codes with one power of two for a block of tokens and a head.
//   s_j = scale * (q . k_j);  o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)   over the tokens j a query sees
// One pass over the tokens with the running maximum m and sum l (in the base-2 exponent: f = scale * log2(e)).
//
// Arithmetic.  Key codes are exact in bf16 and fp16, so q meets them as it is, in q's type; the block's power of two multiplies the
// fp32 score.  The numerators, 2^(s f - m + 6), enter the second product in fp16: m is the largest score until another passes it by 2^8, which
// leaves them below 2^15 and 30 binades above fp16's smallest step.  Value codes are exact in fp16 too; a block's
// power of two is taken relative to the largest, 2^E, of those that a row of the wavefront has seen, so that a value is exact unless its block's is 2^15
// below that, then good to 2^-25 of 2^E.  Where 2^E may be more than 2^8 above the largest that some row of the wavefront sees itself
// (queries at either end of a window, or of a sequence), rows are taken one by one (attend_row), so that values always count to 2^-17 of the largest power
// of two that a query sees.  l sums the numerators as they enter there.  Maxima, sums and results are fp32.
//
// Operands come straight from memory to the matrix instructions, no value crosses lanes between the two products.  The first one
// makes S^T (tokens x queries) from K rows, the second O^T = V^T P^T.  A step has 64 tokens; lane group g (of four) gets scores of tokens
// 16 g .. 16 g + 15 when row 4 a + i of K tile t is token 16 a + 4 t + i, and those are the tokens whose value codes it loads, 16 adjacent bytes
// of a V^T row.
//
// Rows: the queries of a sequence that read one cache head, (token, query head) in turn; 16 rows are the columns of one instruction.
#include <hip/hip_runtime.h>

#include "kv_cache.h"

namespace {

using namespace st_kv;

static_assert(sizeof(st_kv_attention_args) == 208, "the ctypes declaration has this size");

constexpr int kWaves = 4, kThreads = 64 * kWaves, kStep = 64;

// An unfinished result is a sum of numerators times values, in units of 2^(e - 127): its m and l, and e (-1 where l is 0).  A sum in
// units of 1 would pass fp32's range for values above 2^64, whose mean does not.
struct Part {
    float m, l;
    int32_t e;
};

struct Args {
    Seqs s;
    const uint8_t *q, *k, *v, *ks, *vs;
    uint8_t* out;
    float* part;                  // [tokens * query heads][splits][D] unfinished results, or null
    Part* stat;                   // [tokens * query heads][splits]
    uint64_t q_pitch, q_head_pitch, out_pitch, out_head_pitch;
    uint32_t group, causal, window;
    uint32_t tiles, splits;       // row tiles of a head, parts of a tile's tokens at most
    float f;                      // scale * log2(e)
};

constexpr float kNone = -__builtin_inff();
constexpr float kOffset = 6.0f, kSlack = 8.0f;
// Binades below the common power of two in which every value code is exact in fp16; those by which it may be above what a row sees itself (a value is
// good to 2^-25 of the former, then 2^-17 of the latter); and see settle.
constexpr int32_t kNear = 15, kAbove = 8, kRoom = 5;

// The tokens [lo, hi) that row r of a sequence's head sees.
struct Sees {
    int32_t lo, hi;
};
__device__ __forceinline__ Sees sees(const Args& a, const Span& p, uint32_t row) {
    Sees s = {0, p.len};
    if (a.causal) {
        const int32_t pos = p.pos + int32_t(row / a.group);
        if (pos < p.len) s.hi = pos + 1 < 0 ? 0 : pos + 1;
        if (a.window && pos >= int32_t(a.window)) s.lo = pos - int32_t(a.window) + 1;
    }
    return s;
}
// Steps [first, last) that rows row0 .. rows - 1 of a tile need; both ends grow with the row.
struct Steps {
    int32_t first, last;
};
__device__ __forceinline__ Steps steps_of(const Args& a, const Span& p, uint32_t row0, uint32_t end) {
    const int32_t lo = sees(a, p, row0).lo, hi = sees(a, p, end - 1).hi;
    return hi > lo ? Steps{lo / kStep, (hi + kStep - 1) / kStep} : Steps{0, 0};
}

// Steps of each part of a tile: equal ones, four for each wavefront at least.  They follow from the tokens that a tile has, not from those that the
// table has room for, which in a captured graph may be many more.
constexpr uint32_t kLeastPart = 4 * kWaves;
__device__ __forceinline__ uint32_t part_of(const Args& a, const Steps& st) {
    uint32_t part = (uint32_t(st.last - st.first) + a.splits - 1) / a.splits;
    part = (part + kWaves - 1) / kWaves * kWaves;
    return part < kLeastPart ? kLeastPart : part;
}

// Over the four lane groups, by exchanging rows of 16 and halves of 32 lanes on the vector unit.
__device__ __forceinline__ float max_over_groups(float v) {
    auto a = __builtin_amdgcn_permlane16_swap(as_u32(v), as_u32(v), false, false);
    v = fmaxf(as_f32(a[0]), as_f32(a[1]));
    auto b = __builtin_amdgcn_permlane32_swap(as_u32(v), as_u32(v), false, false);
    return fmaxf(as_f32(b[0]), as_f32(b[1]));
}

__device__ __forceinline__ int32_t max_over_groups(int32_t v) {
    auto a = __builtin_amdgcn_permlane16_swap(uint32_t(v), uint32_t(v), false, false);
    v = int32_t(a[0]) > int32_t(a[1]) ? int32_t(a[0]) : int32_t(a[1]);
    auto b = __builtin_amdgcn_permlane32_swap(uint32_t(v), uint32_t(v), false, false);
    return __builtin_amdgcn_readfirstlane(int32_t(b[0]) > int32_t(b[1]) ? int32_t(b[0]) : int32_t(b[1]));
}

// v, as something the compiler knows nothing of: what a rarely taken branch computes from it stays in that branch.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

__device__ __forceinline__ uint32_t opaque_uniform(uint32_t v) {
    asm volatile("" : "+s"(v));
    return v;
}
// The kernel's arguments (its only ones) read again: a rarely taken branch that uses these keeps none of the others in registers through a loop
// ahead of it.
__device__ __forceinline__ Args arguments_again() {
    typedef const __attribute__((address_space(4))) Args* constant;
    uint64_t p = reinterpret_cast<uint64_t>(__builtin_amdgcn_kernarg_segment_ptr());
    asm volatile("" : "+s"(p));
    return *(const Args*)reinterpret_cast<constant>(p);
}

// Bytes of c that are a NaN code (0x7F, 0xFF) as 0xFF.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t c) {
    const uint32_t z = ~(c & 0x7F7F7F7Fu) & 0x7F7F7F7Fu;           // 0 where the code is NaN
    const uint32_t t = (z + 0x7F7F7F7Fu) & 0x80808080u;            // 0x80 where it is not
    return ((t ^ 0x80808080u) >> 7) * 0xFFu;
}

// What a wavefront knows of its 16 * QT rows.
template <bool F16, int D, int QT>
struct Wave {
    static constexpr int KL = D / 64;      // 16-byte loads of a K row per lane
    static constexpr int DT = D / 16;      // 16-column tiles of a result
    u32x4 q[QT][D / 32];
    float m[QT];
    f32x4 l[QT];                           // the sum of a row's numerators, four times, in each of its lanes
    f32x4 o[QT][DT];
    uint32_t nan[QT][(DT + 7) / 8];        // a bit for each result that is NaN whatever o says
    int32_t lo[QT], hi[QT];
    int32_t e = -1;                        // E + 127, -1: no values yet
    int32_t every = -1, low = 256;         // the largest page that every row has seen, a bound below those that some row has (256: none),
    int32_t span = 0;                      // and how far the one is above the other
    int32_t all_lo, all_hi;                // tokens that every row sees
    int32_t any_lo, any_hi;                // tokens that some row sees

    __device__ __forceinline__ void start(const Args& a, const Span& p, uint32_t head, uint32_t row0, uint32_t rows) {
        const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll
        for (int j = 0; j < QT; ++j) {
            const uint32_t row = row0 + 16 * j + r;
            const bool have = row < rows;
            const Sees s = sees(a, p, have ? row : rows - 1);
            lo[j] = s.lo, hi[j] = s.hi;
            const uint32_t t = row / a.group, h = head * a.group + row % a.group;
            const uint8_t* pq = a.q + ((uint64_t(p.first) + (have ? t : 0)) * a.q_pitch + (have ? h : 0) * a.q_head_pitch + D / 4 * g) * 2;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) q[j][c] = have ? u32x4(*reinterpret_cast<const u32x4_any*>(pq + 16 * c)) : u32x4{0, 0, 0, 0};
            m[j] = kNone, l[j] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int d = 0; d < DT; ++d) o[j][d] = f32x4{0, 0, 0, 0}, nan[j][d / 8] = 0;
        }
        const uint32_t last = row0 + 16 * QT < rows ? row0 + 16 * QT : rows;
        const Sees s0 = sees(a, p, row0), s1 = sees(a, p, last - 1);
        all_lo = s1.lo, all_hi = s0.hi, any_lo = s0.lo, any_hi = s1.hi;
    }

    // The common power of two, of lane groups whose 16 tokens some row sees: the pages of others (behind a sequence's end, ahead of a window) may
    // have any.  And what tells whether it serves all rows.
    template <class V>
    __device__ __forceinline__ void settle(int32_t at, uint32_t vs, V v, bool known) {
        const bool none = vs == 255;
        const int32_t now = !none ? int32_t(vs) : e < 0 ? 0 : e;
        const bool some = known && at < any_hi && at + 16 > any_lo, all = some && all_lo < all_hi && at < all_hi && at + 16 > all_lo;
        const int32_t most = max_over_groups(some && now > e ? now : e);
        every = max_over_groups(all && now > every ? now : every);
        bool below = some && !none && now < low;
        if (__any(below)) {
            if (__any(below && now == 0)) {         // pages of zeros, which have the smallest power of two, lose nothing
                uint32_t any = 0;
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const u32x4 c = v(d);
                    any |= c[0] | c[1] | c[2] | c[3];
                }
                below = below && (__ballot(any & 0x7F7F7F7Fu) >> (at & 48) & 0xFFFF) != 0;
            }
            // (with some room, so that pages of ordinary data do not come here one after the other)
            const int32_t least = -max_over_groups(below ? -now : -256);
            if (least < 256) low = least - kRoom;
        }
        span = every > low ? every - low : 0;
        if (most > e) {
            if (e >= 0) {
#pragma unroll
                for (int j = 0; j < QT; ++j)
#pragma unroll
                    for (int d = 0; d < DT; ++d)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[j][d][i] = __builtin_amdgcn_ldexpf(o[j][d][i], e - most);
            }
            e = most;
        }
    }
    // Some row may have seen only pages far below the common power of two, and some page's codes are not exact beside it.
    __device__ __forceinline__ bool apart() const { return low < e - kNear && every < e - kAbove; }

    // One step of tokens from t0.  k(t, i), v(d): its codes, 16 bytes of K tile t and of V^T tile d; ks, vs: the scale codes of lane
    // group g's tokens; known: they lie on a page.  The schedule is cut between tiles, which bounds the registers that decoded
    // codes take.
    template <class K, class V>
    __device__ __forceinline__ void step(const Args& a, int32_t t0, K k, V v, uint32_t ks, uint32_t vs, bool known) {
        const int lane = threadIdx.x & 63, g = lane >> 4;
        f32x4 s[QT][4];
        u32x4 kn[KL];
#pragma unroll
        for (int i = 0; i < KL; ++i) kn[i] = k(0, i);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            u32x4 kc[KL];
#pragma unroll
            for (int i = 0; i < KL; ++i) kc[i] = kn[i];
            if (t + 1 < 4) {
#pragma unroll
                for (int i = 0; i < KL; ++i) kn[i] = k(t + 1, i);
            }
#pragma unroll
            for (int j = 0; j < QT; ++j) s[j][t] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < KL; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const u32x4 kv = codes8<F16, ST_KIND_FP8_TENSOR>(kc[i][2 * h], kc[i][2 * h + 1], 1.0f);
#pragma unroll
                    for (int j = 0; j < QT; ++j) s[j][t] = mfma32<F16>(kv, q[j][2 * i + h], s[j][t]);
                }
            __builtin_amdgcn_sched_barrier(0);
        }
        const float f = power_of(ks) * a.f;
        const bool inside = t0 >= all_lo && t0 + kStep <= all_hi && __all(known);     // every row sees every token
        const int32_t at = t0 + 16 * g;
        u32x4 p[QT][2];
#pragma unroll
        for (int j = 0; j < QT; ++j) {
            // tokens of this lane that the row sees; the scores stay as they are, so that neither case copies them
            const uint32_t from = uint32_t(at - lo[j]), count = known && hi[j] > lo[j] ? uint32_t(hi[j] - lo[j]) : 0;
            float mx = kNone;
            if (inside) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[j][t][i]);
            } else {
                const uint32_t here = opaque(from);
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, here + (4 * t + i) < count ? s[j][t][i] : kNone);
            }
            mx *= mx == kNone ? 1.0f : f;
            mx = max_over_groups(mx);
            if (__any(mx > m[j] + kSlack)) {
                const float now = fmaxf(m[j], mx), keep = now == kNone ? 1.0f : __builtin_amdgcn_exp2f(m[j] - now);
                m[j] = now;
                l[j] *= keep;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[j][d] *= keep;
            }
            const float base = kOffset - (m[j] == kNone ? 0.0f : m[j]);
            if (inside) {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    float x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][t][i], f, base));
                    p[j][t >> 1][2 * (t & 1)] = cvt_f16x2(x[0], x[1]);
                    p[j][t >> 1][2 * (t & 1) + 1] = cvt_f16x2(x[2], x[3]);
                }
            } else {
                const uint32_t here = opaque(from);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    float x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[i] = here + (4 * t + i) < count ? __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][t][i], f, base)) : 0.0f;
                    p[j][t >> 1][2 * (t & 1)] = cvt_f16x2(x[0], x[1]);
                    p[j][t >> 1][2 * (t & 1) + 1] = cvt_f16x2(x[2], x[3]);
                }
            }
            const u32x4 ones = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
            l[j] = mfma32<true>(ones, p[j][1], mfma32<true>(ones, p[j][0], l[j]));
        }
        if (__any(known && vs - uint32_t(low) > uint32_t(span))) settle(at, vs, v, known);
        // (a factor above 1 is one of a page that nobody sees, whose numerators are 0: it must be finite)
        int32_t by = int32_t(vs) - e + 127;
        by = by < 0 ? 0 : by > 127 ? 127 : by;
        const float vf = as_f32(vs == 255 ? 0x7F800000u : uint32_t(by) << 23);
        // Tokens that some rows do not see may hold anything.
        uint32_t found = 0;
        if (!inside) {
            found = vs == 255;
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const u32x4 c = v(d);
                found |= nan_bytes(c[0]) | nan_bytes(c[1]) | nan_bytes(c[2]) | nan_bytes(c[3]);
            }
        }
        const bool dirty = __any(found != 0);
        const uint32_t all = vs == 255 ? 0xFFFFFFFFu : 0;
        if (dirty) {
            // NaN codes are taken out below, and the results of the rows that see them noted here: the code of 1 (0x38) in their place
            // times 1 where the row sees the token
#pragma unroll
            for (int j = 0; j < QT; ++j) {
                const uint32_t from = uint32_t(at - lo[j]), count = known && hi[j] > lo[j] ? uint32_t(hi[j] - lo[j]) : 0;
                u32x4 y[2];
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    y[t >> 2][t & 3] = (from + 2 * t < count ? 0x3C00u : 0u) | (from + 2 * t + 1 < count ? 0x3C000000u : 0u);
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    u32x4 b = v(d);
#pragma unroll
                    for (int w = 0; w < 4; ++w) b[w] = (nan_bytes(b[w]) | all) & 0x38383838u;
                    const u32x4 b0 = codes8<true, ST_KIND_FP8_TENSOR>(b[0], b[1], 1.0f), b1 = codes8<true, ST_KIND_FP8_TENSOR>(b[2], b[3], 1.0f);
                    const f32x4 hit = mfma32<true>(b1, y[1], mfma32<true>(b0, y[0], f32x4{0, 0, 0, 0}));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (hit[i] > 0.0f) nan[j][d / 8] |= 1u << (d % 8 * 4 + i);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        const float vm = dirty && vs == 255 ? 1.0f : vf;
        u32x4 vn = v(0);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            u32x4 c = vn;
            if (d + 1 < DT) vn = v(d + 1);
            if (dirty) {
#pragma unroll
                for (int w = 0; w < 4; ++w) c[w] &= ~(nan_bytes(c[w]) | all);
            }
            const u32x4 v0 = codes8<true, ST_KIND_FP8_TENSOR>(c[0], c[1], vm), v1 = codes8<true, ST_KIND_FP8_TENSOR>(c[2], c[3], vm);
#pragma unroll
            for (int j = 0; j < QT; ++j) o[j][d] = mfma32<true>(v0, p[j][0], o[j][d]);
#pragma unroll
            for (int j = 0; j < QT; ++j) o[j][d] = mfma32<true>(v1, p[j][1], o[j][d]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // The exponent of a row's units.
    __device__ __forceinline__ int32_t units(int j) const { return l[j][0] == 0.0f ? -1 : e; }
    // o times a factor of the row's and 2^up
    __device__ __forceinline__ f32x4 result(int j, int d, float by, int32_t up) const {
        f32x4 x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = __builtin_amdgcn_ldexpf(o[j][d][i] * by, up);
            if (nan[j][d / 8] >> (d % 8 * 4 + i) & 1) x[i] = __builtin_nanf("");
        }
        return x;
    }
};

// Four consecutive results of one row to the output.
template <bool F16>
__device__ __forceinline__ void store_row4(const Args& a, uint64_t i, const float* v) {
    const uint32_t lo = F16 ? cvt_f16x2(v[0], v[1]) : cvt_bf16x2(v[0], v[1]), hi = F16 ? cvt_f16x2(v[2], v[3]) : cvt_bf16x2(v[2], v[3]);
    *reinterpret_cast<u64_any*>(a.out + i * 2) = uint64_t(hi) << 32 | lo;
}

// What a workgroup has: rows row0 .. end - 1 of a sequence's head, over the steps st.
struct Tile {
    uint32_t seq, head, row0, end, rows, split;
    Span p;
    Steps st;
};
// The rest of t from its sequence, head, row0 and split; false: nothing to do.
__device__ __forceinline__ bool complete(const Args& a, uint32_t tile_rows, Tile& t) {
    t.p = span_of(a.s, t.seq);
    t.rows = uint32_t(t.p.count) * a.group;
    if (t.row0 >= t.rows) return false;
    t.end = t.row0 + tile_rows < t.rows ? t.row0 + tile_rows : t.rows;
    t.st = steps_of(a, t.p, t.row0, t.end);
    if (a.splits > 1) {
        const uint32_t part = part_of(a, t.st);
        t.st.first += int32_t(t.split * part);
        if (t.st.first >= t.st.last) return false;
        t.st.last = t.st.first + int32_t(part) < t.st.last ? t.st.first + int32_t(part) : t.st.last;
    }
    return true;
}
__device__ __forceinline__ bool tile_of(const Args& a, uint32_t tile_rows, uint32_t block, Tile& t) {
    // All first parts, then all second ones, and so on: those that sequences do not have leave no gaps between the others, which would come in patterns
    // that idle part of the XCDs (16 sequences' 4 drafts, 64 queries on 8 heads of 128: 74 us, and with a table 16 times as wide as the
    // longest; 92 and 168 with a tile's parts one after the other).  Tiles of a head, which read the same codes, close together, after
    // the heads (32 sequences' 16 drafts, 32 queries on 8 heads of 64: 64 us; 67 with tiles ahead of heads, 74 behind sequences).
    t.head = block % a.s.heads;
    block /= a.s.heads;
    t.row0 = block % a.tiles * tile_rows;
    block /= a.tiles;
    t.seq = block % a.s.seqs, t.split = block / a.s.seqs;
    return complete(a, tile_rows, t);
}

// One row of a tile by one wavefront, its own numerators and powers of two in fp32: for rows that a power of two in common does not
// serve (Wave::apart()).  A lane has one token's score, then D / 64 results.  Simple rather than fast, since pages of one sequence and head do not differ
// like that in earnest: 4 prompts' chunks of up to 2048 tokens, 32 heads of 128, through windows of 300 take 1.96 ms where each page's values are 2^12
// below those of the one before, 0.10 where they are not.
template <bool F16, int D>
__device__ __forceinline__ void attend_row(const Args& a, const Tile& tile, uint32_t row) {
    const Span& p = tile.p;
    const uint32_t seq = tile.seq, head = tile.head, split = tile.split;
    const Steps st = tile.st;
    constexpr int COLS = D / 64;
    const int lane = threadIdx.x & 63;
    const uint32_t bl = a.s.block_log2, block = 1u << bl;
    const uint64_t page_bytes = uint64_t(block) * D, tok = uint64_t(p.first) + row / a.group, h = head * a.group + row % a.group;
    const uint8_t* q = a.q + (tok * a.q_pitch + h * a.q_head_pitch) * 2;
    const Sees see = sees(a, p, row);
    float m = kNone, l = 0.0f, o[COLS];
    int32_t e = -1;
#pragma unroll
    for (int c = 0; c < COLS; ++c) o[c] = 0.0f;
    for (int32_t i = st.first; i < st.last; ++i) {
        const int32_t t0 = i * kStep, t = t0 + lane;
        const int32_t page = page_of(a.s, seq, int64_t(t) >> bl);
        const uint64_t at = uint64_t(page < 0 ? 0 : page) * a.s.heads + head;
        const bool seen = page >= 0 && t >= see.lo && t < see.hi;
        float s = kNone;
        if (seen) {
            const uint8_t* k = a.k + at * page_bytes + uint64_t(t & (block - 1)) * D;
            s = 0.0f;
#pragma unroll 8
            for (int c = 0; c < D; c += 4) {
                const uint32_t code = *reinterpret_cast<const uint32_t*>(k + c);
                const uint64_t x = *reinterpret_cast<const u64_any*>(q + 2 * c);
                const f32x2 k0 = __builtin_amdgcn_cvt_pk_f32_fp8(code, false), k1 = __builtin_amdgcn_cvt_pk_f32_fp8(code, true);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const uint32_t u = uint32_t(x >> 16 * n) & 0xFFFF;
                    const float f = F16 ? float(__builtin_bit_cast(f16x2, u).x) : as_f32(u << 16);
                    s = __builtin_fmaf(n < 2 ? k0[n] : k1[n - 2], f, s);
                }
            }
            s *= power_of(a.ks[at]) * a.f;
        }
        float top = s;
#pragma unroll
        for (int x = 1; x < 64; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
        const float now = fmaxf(m, top), keep = now == kNone ? 1.0f : __builtin_amdgcn_exp2f(m - now);
        m = now, l *= keep;
        const float n = seen ? __builtin_amdgcn_exp2f(s + (kOffset - (m == kNone ? 0.0f : m))) : 0.0f;
        float sum = n;
#pragma unroll
        for (int x = 1; x < 64; x *= 2) sum += __shfl_xor(sum, x);
        l += sum;
#pragma unroll
        for (int c = 0; c < COLS; ++c) o[c] *= keep;
        const uint64_t mask = __ballot(seen);
#pragma unroll 1
        for (int g = 0; g < 64; g += 16) {
            if (!(mask >> g & 0xFFFF)) continue;
            const uint64_t of = uint64_t(__builtin_amdgcn_readlane(page, g)) * a.s.heads + head;
            const uint8_t* v = a.v + of * page_bytes + uint64_t(lane) * COLS * block + ((t0 + g) & (block - 1));
            const int32_t code = a.vs[of], unit = code == 255 ? 0 : code, to = unit > e ? unit : e;
            const float by = code == 255 ? __builtin_nanf("") : 1.0f;
            float x[COLS];
#pragma unroll
            for (int c = 0; c < COLS; ++c) x[c] = 0.0f;
#pragma unroll 1
            for (int b = g; b < g + 16; b += 4) {
                // (what tokens that the row does not see hold may be NaN)
                const uint32_t in = (uint32_t(mask >> b & 15) * 0x204081u & 0x01010101u) * 0xFFu;
#pragma unroll
                for (int c = 0; c < COLS; ++c) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(v + uint64_t(c) * block + (b - g)) & in;
                    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
                    const float value[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
                    for (int t = 0; t < 4; ++t) x[c] = __builtin_fmaf(as_f32(__builtin_amdgcn_readlane(as_u32(n), b + t)), value[t], x[c]);
                }
            }
#pragma unroll
            for (int c = 0; c < COLS; ++c) o[c] = __builtin_amdgcn_ldexpf(o[c], e - to) + __builtin_amdgcn_ldexpf(x[c] * by, unit - to);
            e = to;
        }
    }
    if (l == 0.0f) e = -1;
    const uint64_t out = tok * a.s.heads * a.group + h;
    if (a.splits > 1 && lane == 0) a.stat[out * a.splits + split] = Part{m, l, e};
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
        const uint32_t d = lane * COLS + c;
        if (a.splits > 1) {
            a.part[(out * a.splits + split) * D + d] = o[c];
        } else {
            const float y = l == 0.0f ? 0.0f : __builtin_amdgcn_ldexpf(o[c] / l, e - 127);
            *reinterpret_cast<uint16_t*>(a.out + (tok * a.out_pitch + h * a.out_head_pitch + d) * 2) = uint16_t(F16 ? cvt_f16x2(y, 0.0f) : cvt_bf16x2(y, 0.0f));
        }
    }
}

// Few rows: the wavefronts of a workgroup take the steps of one row tile in turn and join in LDS, in their order.  Bound by the codes' bytes: one
// query of 2 sequences of 131071 tokens, 8 heads of 128 and five queries each (537 MB), 111 us, 4.8 TB/s; of 48 sequences of 100 to 8192 tokens
// (408 MB) 94 to 97 us, 4.3 TB/s, whether the table holds the longest or 131072 tokens.  3 sequences' 4 drafts, 8 heads of 64, up to 1000
// tokens: 9 us, of which the launch and four dependent loads (length, page, codes, scale) are most.
template <bool F16, int D, int QT>
__global__ __launch_bounds__(kThreads, D * QT <= 128 ? 2 : 1) void attend(Args a) {
    using W = Wave<F16, D, QT>;
    constexpr int ROWS = 16 * QT, PITCH = D + 4;
    __shared__ __align__(16) float sum[ROWS][PITCH];
    __shared__ float top[kWaves][ROWS], den[kWaves][ROWS];
    __shared__ int32_t unit[kWaves][ROWS], apart[kWaves];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Tile t;
    if (!tile_of(a, ROWS, blockIdx.x, t)) return;
    const Span p = t.p;
    const Steps st = t.st;
    const uint32_t seq = t.seq, head = t.head, row0 = t.row0, end = t.end, rows = t.rows, split = t.split;
    W w;
    w.start(a, p, head, row0, rows);

    const uint32_t bl = a.s.block_log2, block = 1u << bl;
    const uint64_t page_bytes = uint64_t(block) * D;
    u32x4 k[4][W::KL], v[W::DT];
    uint32_t ks = 0, vs = 0;
    bool known = false;
    // the pages of step i's tokens: of the K rows this lane loads, and of its group's
    auto pages = [&](int32_t i, int32_t& pk, int32_t& pv) {
        pk = page_of(a.s, seq, (int64_t(i) * kStep + 16 * (r >> 2)) >> bl);
        pv = page_of(a.s, seq, (int64_t(i) * kStep + 16 * g) >> bl);
    };
    auto load_k = [&](int32_t i, int32_t pk) {
        const uint64_t at = (uint64_t(pk < 0 ? 0 : pk) * a.s.heads + head) * page_bytes;
        const uint8_t* base = a.k + at + uint64_t(((i * kStep + 16 * (r >> 2)) & (block - 1)) + (r & 3)) * D + D / 4 * g;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int h = 0; h < W::KL; ++h) k[t][h] = *reinterpret_cast<const u32x4*>(base + t * 4 * D + 16 * h);
    };
    auto load_v = [&](int32_t i, int32_t pv) {
        const uint64_t at = uint64_t(pv < 0 ? 0 : pv) * a.s.heads + head;
        const uint8_t* base = a.v + at * page_bytes + uint64_t(r) * block + ((i * kStep + 16 * g) & (block - 1));
#pragma unroll
        for (int d = 0; d < W::DT; ++d) v[d] = *reinterpret_cast<const u32x4*>(base + uint64_t(d * 16) * block);
        known = pv >= 0;
        ks = known ? a.ks[at] : 0, vs = known ? a.vs[at] : 0;
    };
    int32_t i = st.first + wave, pk, pv;
    if (i < st.last) {
        pages(i, pk, pv);
        load_k(i, pk);
        load_v(i, pv);
        for (; i < st.last; i += kWaves) {
            w.step(a, i * kStep, [&](int t, int h) { return k[t][h]; }, [&](int d) { return v[d]; }, ks, vs, known);
            if (i + kWaves < st.last) {
                pages(i + kWaves, pk, pv);
                load_k(i + kWaves, pk);
                load_v(i + kWaves, pv);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < QT; ++j) {
        if (g == 0) top[wave][16 * j + r] = w.m[j], den[wave][16 * j + r] = w.l[j][0], unit[wave][16 * j + r] = w.units(j);
    }
    if (lane == 0) apart[wave] = w.apart();
    __syncthreads();
    if (apart[0] | apart[1] | apart[2] | apart[3]) {
        const Args b = arguments_again();
        if (!tile_of(b, ROWS, opaque_uniform(blockIdx.x), t)) return;
        for (uint32_t row = t.row0 + wave; row < t.end; row += kWaves) attend_row<F16, D>(b, t, row);
        return;
    }
    float m[QT];
#pragma unroll
    for (int j = 0; j < QT; ++j) {
        m[j] = kNone;
        int32_t e = -1;
#pragma unroll
        for (int o = 0; o < kWaves; ++o) {
            m[j] = fmaxf(m[j], top[o][16 * j + r]);
            e = unit[o][16 * j + r] > e ? unit[o][16 * j + r] : e;
        }
        const float keep = w.m[j] == kNone ? 1.0f : __builtin_amdgcn_exp2f(w.m[j] - m[j]);
#pragma unroll
        for (int d = 0; d < W::DT; ++d) w.o[j][d] = w.result(j, d, keep, w.units(j) - e);
    }
#pragma unroll
    for (int o = 0; o < kWaves; ++o) {
        if (wave == o) {
#pragma unroll
            for (int j = 0; j < QT; ++j)
#pragma unroll
                for (int d = 0; d < W::DT; ++d) {
                    f32x4* at = reinterpret_cast<f32x4*>(&sum[16 * j + r][16 * d + 4 * g]);
                    *at = o == 0 ? w.o[j][d] : *at + w.o[j][d];
                }
        }
        __syncthreads();
    }
    for (uint32_t i4 = threadIdx.x; i4 < (end - row0) * (D / 4); i4 += kThreads) {
        const uint32_t rr = i4 / (D / 4), d = i4 % (D / 4) * 4, row = row0 + rr;
        float m1 = kNone, l = 0.0f;
        int32_t e = -1;
#pragma unroll
        for (int o = 0; o < kWaves; ++o) m1 = fmaxf(m1, top[o][rr]), e = unit[o][rr] > e ? unit[o][rr] : e;
#pragma unroll
        for (int o = 0; o < kWaves; ++o) l += top[o][rr] == kNone ? den[o][rr] : den[o][rr] * __builtin_amdgcn_exp2f(top[o][rr] - m1);
        f32x4 x = *reinterpret_cast<const f32x4*>(&sum[rr][d]);
        const uint64_t tok = uint64_t(p.first) + row / a.group, h = head * a.group + row % a.group;
        if (a.splits > 1) {
            const uint64_t at = (tok * a.s.heads * a.group + h) * a.splits + split;
            *reinterpret_cast<f32x4*>(a.part + at * D + d) = x;
            if (d == 0) a.stat[at] = Part{m1, l, e};
        } else {
            float y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) y[c] = l == 0.0f ? 0.0f : __builtin_amdgcn_ldexpf(x[c] / l, e - 127);
            store_row4<F16>(a, tok * a.out_pitch + h * a.out_head_pitch + d, y);
        }
    }
}

// Many rows, bound by issuing: for 64 tokens of 32 rows and heads of 128 a wavefront has 64 + 4 matrix instructions of 16 cycles, and
// decodes codes (4 cycles a pair) and takes exponentials (8 cycles each) on the vector unit for 1.7 times as long, which another wavefront's
// matrix instructions hide in part.  The last (682, 2048, 1365, 1) of (3466, 6200, 4833, 2100) tokens, 8 heads of 128 and four queries each
// (301 GFLOP): 440 us, 690 TFLOP/s.
// Four wavefronts of 16 * QT rows each share the codes of a step, which go from memory straight to LDS, kStages - 1 steps ahead.
// LDS holds rows of 16-byte chunks, K's in the order of the instructions' rows (row 16 t + r: the token that lane r has in K tile
// t), V^T's as they are; chunk c of a row sits at c ^ swizzle(row), so that 16 lanes reading one chunk of 16 rows touch all banks once.
constexpr int kStages = 3;
template <int CHUNKS>
__device__ __forceinline__ int swizzle(int row) {
    return CHUNKS == 4 ? (row >> 2) & 3 : CHUNKS == 8 ? (row >> 1) & 7 : row & 15;
}
__device__ __forceinline__ void to_lds16(const uint8_t* from, uint8_t* to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from, (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}
// s_waitcnt for vmcnt(n) and lgkmcnt(0), expcnt at its maximum (gfx9 encoding: vmcnt in bits 3:0 and 15:14)
constexpr int wait_vmem(int n) { return (n & 15) | (n >> 4) << 14 | 7 << 4; }

// The sequence, head and row tile of this workgroup.  Workgroup b runs on XCD b mod 8.  An XCD takes an eighth of the heads, or with 8 / n
// others every so-many-th tile of one of n heads, so that a head's codes meet in its L2; the longest sequences come first, and of each
// the tiles with the most tokens.  There is no gap between the tiles of sequences of different size: workgroups without
// work would come in patterns that leave part of an XCD idle (4 prompts' chunks, as above: 1.7 times as long with gaps between the longest's tiles).
// All lanes of a wavefront take part, 64 sequences at a time.
template <int ROWS>
__device__ __forceinline__ bool place(const Args& a, uint32_t block, Tile& to) {
    const uint32_t H = a.s.heads, lane = threadIdx.x & 63, xcd = block % 8;
    const uint32_t ways = H % 8 == 0 ? 1 : 8 % H == 0 ? 8 / H : 8, groups = 8 / ways, per = H % 8 == 0 ? H / 8 : 8 % H == 0 ? 1 : H;
    const uint32_t way = xcd / groups;
    uint32_t at = block / 8 / a.splits;
    to.split = block / 8 % a.splits;
    for (uint32_t base = 0; base < a.s.seqs; base += 64) {
        const uint32_t s = base + lane;
        uint32_t tiles = 0, len = 0;
        if (s < a.s.seqs) {
            const Span p = span_of(a.s, s);
            const uint32_t all = (uint32_t(p.count) * a.group + ROWS - 1) / ROWS;
            tiles = all > way ? (all - way + ways - 1) / ways : 0;
            len = uint32_t(p.len);
        }
        uint32_t before = 0, total = 0;
        const uint32_t n = a.s.seqs - base < 64 ? a.s.seqs - base : 64;
        for (uint32_t o = 0; o < n; ++o) {
            const uint32_t t = __builtin_amdgcn_readlane(tiles, o), l = __builtin_amdgcn_readlane(len, o);
            before += l > len || (l == len && o < lane) ? t : 0;
            total += t;
        }
        if (at < total * per) {
            const uint64_t hit = __ballot(at >= before * per && at < (before + tiles) * per);
            const uint32_t o = uint32_t(__builtin_ctzll(hit)), t = __builtin_amdgcn_readlane(tiles, o);
            at -= __builtin_amdgcn_readlane(before, o) * per;
            to.seq = base + o;
            to.head = xcd % groups + (per > 1 ? at / t * groups : 0);
            to.row0 = (way + (t - 1 - at % t) * ways) * ROWS;
            return complete(a, ROWS, to);
        }
        at -= total * per;
    }
    return false;
}

template <bool F16, int D, int QT>
__global__ __launch_bounds__(kThreads, D * QT <= 256 ? 2 : 1) void attend_many(Args a) {
    using W = Wave<F16, D, QT>;
    constexpr int ROWS = 16 * QT * kWaves, KC = D / 16, KB = kStep * D, STAGE = 2 * KB;
    constexpr int PER = KB / 16 / kThreads;           // chunks of K, and of V, per thread and step
    constexpr int PITCH = D + 4;
    constexpr int OUT = kWaves * 16 * PITCH * 4, LDS = kStages * STAGE > OUT ? kStages * STAGE : OUT;
    static_assert(PER >= 1, "a chunk for each thread");
    __shared__ __align__(128) uint8_t lds[LDS];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Tile t;
    if (!place<ROWS>(a, blockIdx.x, t)) return;
    const Span p = t.p;
    const Steps st = t.st;
    const uint32_t seq = t.seq, head = t.head, row0 = t.row0, end = t.end, rows = t.rows, split = t.split;
    const uint32_t mine = row0 + wave * 16 * QT;
    const bool work = mine < end;
    W w;
    w.start(a, p, head, work ? mine : row0, rows);

    const uint32_t bl = a.s.block_log2, block = 1u << bl;
    const uint64_t page_bytes = uint64_t(block) * D;
    // Lane l keeps the page of the l-th 16 tokens of 16 steps, and its scales; the next 16 steps' are on their way.
    int32_t page = 0, next_page = 0;
    uint32_t scales = 0, next_scales = 0;         // ks | vs << 8
    auto fetch_page = [&](int32_t step) { return page_of(a.s, seq, (int64_t(step) * kStep + 16 * lane) >> bl); };
    auto fetch_scales = [&](int32_t pg) {
        const uint64_t at = uint64_t(pg < 0 ? 0 : pg) * a.s.heads + head;
        return pg < 0 ? 0u : uint32_t(a.ks[at]) | uint32_t(a.vs[at]) << 8;
    };
    auto from_lane = [](uint32_t v, int l) { return uint32_t(__builtin_amdgcn_ds_bpermute(l * 4, int(v))); };
    // this thread's chunks: K row 16 t + kr (t = its turn), V^T column block vg of rows tid / 4 + ...
    const int kslot = tid % KC, krow = tid / KC, kr = krow % 16, kg = kr >> 2;
    const int vg = (tid % 4) ^ swizzle<4>(tid / 4);
    const int32_t pages_at = st.first;
    auto issue = [&](int32_t step, int buf, int32_t pg, int32_t base) {
        const int l = (step - base) * 4;
        const int32_t pk = int32_t(from_lane(uint32_t(pg), l + kg)), pv = int32_t(from_lane(uint32_t(pg), l + vg));
        const uint8_t* fk = a.k + (uint64_t(pk < 0 ? 0 : pk) * a.s.heads + head) * page_bytes + uint64_t((step * kStep + 16 * kg) & (block - 1)) * D;
        const uint8_t* fv = a.v + (uint64_t(pv < 0 ? 0 : pv) * a.s.heads + head) * page_bytes + ((step * kStep + 16 * vg) & (block - 1));
        uint8_t* to = lds + buf * STAGE + wave * 1024;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int row = i * (kThreads / KC) + krow, t = row / 16;
            to_lds16(fk + (4 * t + (kr & 3)) * D + (kslot ^ swizzle<KC>(row)) * 16, to + i * (kThreads * 16));
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            to_lds16(fv + uint64_t(i * (kThreads / 4) + tid / 4) * block, to + KB + i * (kThreads * 16));
    };
    const int32_t count = st.last - st.first;
    if (count > 0) {
        page = fetch_page(st.first);
        next_page = fetch_page(st.first + 16);
        scales = fetch_scales(page);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i)
            if (i < count) issue(st.first + i, i, page, pages_at);
    }
    int32_t base = pages_at;
    int buf = 0;
    for (int32_t i = 0; i < count; ++i) {
        const int32_t step = st.first + i;
        if (step - base == 16) {
            base = step, page = next_page, scales = next_scales;
            next_page = fetch_page(base + 16);
        }
        if (step - base == 4) next_scales = fetch_scales(next_page);
        // this step's codes are in LDS and nobody reads the buffer that is filled next
        if (i + 1 < count) __builtin_amdgcn_s_waitcnt(wait_vmem((kStages - 2) * 2 * PER));
        else __builtin_amdgcn_s_waitcnt(wait_vmem(0));
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "singlethread");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "singlethread");
        if (i + kStages - 1 < count) {
            const int32_t s2 = step + kStages - 1;
            const bool on = s2 - base < 16;
            issue(s2, buf + kStages - 1 < kStages ? buf + kStages - 1 : buf - 1, on ? page : next_page, on ? base : base + 16);
        }
        const int32_t t0 = step * kStep;
        if (work && t0 < w.any_hi && t0 + kStep > w.any_lo) {
            const uint8_t* sk = lds + buf * STAGE;
            auto k = [&](int t, int h) {
                return *reinterpret_cast<const u32x4*>(sk + (16 * t + r) * D + ((W::KL * g + h) ^ swizzle<KC>(16 * t + r)) * 16);
            };
            auto v = [&](int d) { return *reinterpret_cast<const u32x4*>(sk + KB + (16 * d + r) * kStep + (g ^ swizzle<4>(16 * d + r)) * 16); };
            const int l = (step - base) * 4 + g;
            const bool known = int32_t(from_lane(uint32_t(page), l)) >= 0;
            const uint32_t sc = from_lane(scales, l);
            w.step(a, t0, k, v, sc & 0xFF, sc >> 8, known);
        }
        buf = buf + 1 < kStages ? buf + 1 : 0;
    }
    __syncthreads();
    if (work && w.apart()) {
        const Args b = arguments_again();
        if (!place<ROWS>(b, opaque_uniform(blockIdx.x), t)) return;
        const uint32_t first = t.row0 + wave * 16 * QT;
        for (uint32_t row = first; row < first + 16 * QT && row < t.end; ++row) attend_row<F16, D>(b, t, row);
        return;
    }
    float* mem = reinterpret_cast<float*>(lds) + wave * 16 * PITCH;
#pragma unroll
    for (int j = 0; j < QT; ++j) {
        const float l = w.l[j][0];
        const float inv = a.splits > 1 ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
        const int32_t e = w.units(j), up = a.splits > 1 || e < 0 ? 0 : e - 127;
#pragma unroll
        for (int d = 0; d < W::DT; ++d) *reinterpret_cast<f32x4*>(mem + r * PITCH + 16 * d + 4 * g) = w.result(j, d, inv, up);
        const uint32_t first = mine + 16 * j;
        if (a.splits > 1 && g == 0 && first + r < end) {
            const uint32_t row = first + r;
            const uint64_t at = ((uint64_t(p.first) + row / a.group) * a.s.heads * a.group + head * a.group + row % a.group) * a.splits + split;
            a.stat[at] = Part{w.m[j], l, e};
        }
#pragma unroll 1
        for (int i4 = lane; i4 < 16 * (D / 4); i4 += 64) {
            const uint32_t row = first + i4 / (D / 4), d = i4 % (D / 4) * 4;
            if (row >= end) break;
            const f32x4 x = *reinterpret_cast<const f32x4*>(mem + i4 / (D / 4) * PITCH + d);
            const uint64_t tok = uint64_t(p.first) + row / a.group, h = head * a.group + row % a.group;
            if (a.splits > 1) {
                *reinterpret_cast<f32x4*>(a.part + ((tok * a.s.heads * a.group + h) * a.splits + split) * D + d) = x;
            } else {
                const float y[4] = {x[0], x[1], x[2], x[3]};
                store_row4<F16>(a, tok * a.out_pitch + h * a.out_head_pitch + d, y);
            }
        }
    }
}

// The parts of rows: D / 4 lanes hold a result; `ways` such groups of lanes share a row, each taking every so-many-th part, and join in LDS,
// all in the parts' order.  (A whole workgroup for a row of two parts would take longer than the attention: 32 sequences' 16 drafts, 32
// heads of 64.)
template <bool F16, int D>
__global__ __launch_bounds__(kThreads) void join(Args a, uint32_t tile_rows, uint32_t ways) {
    constexpr uint32_t LANES = D / 4, GROUPS = kThreads / LANES;
    __shared__ __align__(16) float sum[GROUPS][D];
    __shared__ float top[GROUPS], den[GROUPS];
    __shared__ int32_t unit[GROUPS];
    const uint32_t heads = a.s.heads * a.group, seq = blockIdx.y;
    const Span p = span_of(a.s, seq);
    const uint32_t d = threadIdx.x % LANES * 4, mine = threadIdx.x / LANES, way = mine % ways;
    const uint64_t item = uint64_t(blockIdx.x) * (GROUPS / ways) + mine / ways;
    const uint32_t t = uint32_t(item / heads), h = uint32_t(item % heads);
    const bool have = t < uint32_t(p.count);
    const uint64_t at = ((uint64_t(p.first) + t) * heads + h) * a.splits;
    float m = kNone, l = 0.0f;
    int32_t e = -1;
    f32x4 x = {0, 0, 0, 0};
    auto scaled = [](f32x4 v, float by, int32_t up) {
        v *= by;
        return f32x4{__builtin_amdgcn_ldexpf(v[0], up), __builtin_amdgcn_ldexpf(v[1], up), __builtin_amdgcn_ldexpf(v[2], up), __builtin_amdgcn_ldexpf(v[3], up)};
    };
    if (have) {
        const uint32_t rows = uint32_t(p.count) * a.group, row = t * a.group + h % a.group, row0 = row / tile_rows * tile_rows;
        const Steps st = steps_of(a, p, row0, row0 + tile_rows < rows ? row0 + tile_rows : rows);
        const uint32_t part = part_of(a, st), parts = (uint32_t(st.last - st.first) + part - 1) / part;
        const uint32_t n = parts > way ? (parts - way + ways - 1) / ways : 0;      // (a loop the compiler can unroll: it would wait for each load)
#pragma unroll 4
        for (uint32_t i = 0; i < n; ++i) {
            const Part s = a.stat[at + way + i * ways];
            m = fmaxf(m, s.m);
            e = s.e > e ? s.e : e;
        }
#pragma unroll 4
        for (uint32_t i = 0; i < n; ++i) {
            const uint64_t o = at + way + i * ways;
            const Part s = a.stat[o];
            const float keep = s.m == kNone ? 1.0f : __builtin_amdgcn_exp2f(s.m - m);
            l += s.l * keep;
            x += scaled(*reinterpret_cast<const f32x4*>(a.part + o * D + d), keep, s.e - e);
        }
    }
    if (ways > 1) {
        *reinterpret_cast<f32x4*>(&sum[mine][d]) = x;
        if (d == 0) top[mine] = m, den[mine] = l, unit[mine] = e;
        __syncthreads();
        if (way != 0) return;
        for (uint32_t o = 1; o < ways; ++o) m = fmaxf(m, top[mine + o]), e = unit[mine + o] > e ? unit[mine + o] : e;
        l = 0.0f, x = f32x4{0, 0, 0, 0};
        for (uint32_t o = 0; o < ways; ++o) {
            const float keep = top[mine + o] == kNone ? 1.0f : __builtin_amdgcn_exp2f(top[mine + o] - m);
            l += den[mine + o] * keep;
            x += scaled(*reinterpret_cast<const f32x4*>(&sum[mine + o][d]), keep, unit[mine + o] - e);
        }
    }
    if (!have) return;
    float y[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = l == 0.0f ? 0.0f : __builtin_amdgcn_ldexpf(x[c] / l, e - 127);
    store_row4<F16>(a, (uint64_t(p.first) + t) * a.out_pitch + uint64_t(h) * a.out_head_pitch + d, y);
}

// ------------------------------------------------------------------------- host

const char* kWho = "st_kv_attention";

bool off(const void* p, uint64_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

struct Plan {
    uint64_t rows;               // of a sequence's head, at most
    uint32_t qt, tile_rows, tiles, splits;
    uint64_t count;              // new tokens of a sequence, at most
    bool many;
    uint32_t positions;          // workgroups of an XCD, at most
    uint64_t part_bytes, stat_bytes;
};

st_status check_args(const st_kv_attention_args* g) {
    if (!g) return st_fail(ST_E_ARG, "%s: null arguments", kWho);
    if (g->q_type > ST_OUT_F16) return st_fail(ST_E_ARG, "%s: q type %u is not bf16 or fp16", kWho, g->q_type);
    if (!(g->scale > 0.0 && g->scale < 1e30)) return st_fail(ST_E_ARG, "%s: scale %g is not positive", kWho, g->scale);
    if (g->causal > 1) return st_fail(ST_E_ARG, "%s: causal is %u", kWho, g->causal);
    if (g->window && !g->causal) return st_fail(ST_E_ARG, "%s: a window needs causal attention", kWho);
    if (g->head_dim != 64 && g->head_dim != 128 && g->head_dim != 256)
        return st_fail(ST_E_SHAPE, "%s: head_dim %u is not 64, 128 or 256", kWho, g->head_dim);
    if (g->block != 16 && g->block != 32 && g->block != 64 && g->block != 128)
        return st_fail(ST_E_SHAPE, "%s: block %u is not 16, 32, 64 or 128", kWho, g->block);
    const uint64_t lim = uint64_t(1) << 31;
    if (g->tokens >= lim || g->max_new >= lim || g->pages >= lim || g->table_blocks >= lim / 2 / g->block || g->seqs > 65535 ||
        g->heads > 65535 || g->group > 65535)
        return st_fail(ST_E_SHAPE, "%s: %llu tokens, %llu sequences, %u heads of %u, %llu pages or %llu blocks a sequence are too many",
                       kWho, (unsigned long long)g->tokens, (unsigned long long)g->seqs, g->heads, g->group,
                       (unsigned long long)g->pages, (unsigned long long)g->table_blocks);
    if (g->tokens == 0 || g->seqs == 0 || g->heads == 0 || g->group == 0) return ST_OK;
    if (g->tokens * g->heads >= (uint64_t(1) << 40) / g->group)
        return st_fail(ST_E_SHAPE, "%s: %llu tokens of %u times %u heads are too many", kWho, (unsigned long long)g->tokens, g->heads, g->group);
    if (!g->starts && g->tokens % g->seqs)
        return st_fail(ST_E_SHAPE, "%s: %llu tokens are not %llu equal parts", kWho, (unsigned long long)g->tokens, (unsigned long long)g->seqs);
    if (g->pages == 0 || g->table_blocks == 0) return st_fail(ST_E_SHAPE, "%s: a cache without pages", kWho);
    if (!g->q || !g->out || !g->k || !g->v || !g->k_scale || !g->v_scale || !g->table || !g->lengths)
        return st_fail(ST_E_ARG, "%s: null pointer", kWho);
    if (g->seqs > 1 && g->table_pitch < g->table_blocks) return st_fail(ST_E_SHAPE, "%s: the table's pitch is shorter than its row", kWho);
    if (off(g->q, 2) || off(g->out, 2)) return st_fail(ST_E_ARG, "%s: a pointer is not aligned to its element type", kWho);
    if (off(g->k, 16) || off(g->v, 16)) return st_fail(ST_E_ARG, "%s: the cache is not 16-byte aligned", kWho);
    if (off(g->table, 4) || off(g->lengths, 4) || off(g->starts, 4)) return st_fail(ST_E_ARG, "%s: a table is not 4-byte aligned", kWho);
    return ST_OK;
}

st_status plan_of(const st_kv_attention_args& g, Plan* p) {
    *p = Plan{};
    uint64_t count = g.max_new < g.tokens ? g.max_new : g.tokens;
    if (!g.starts && g.tokens / g.seqs < count) count = g.tokens / g.seqs;
    p->rows = count * g.group;
    if (p->rows == 0) return ST_OK;
    if (p->rows >= uint64_t(1) << 31) return st_fail(ST_E_SHAPE, "%s: %llu queries of a head are too many", kWho, (unsigned long long)p->rows);
    p->count = count;
    // Sharing a step's codes in LDS costs its barriers and fewer, larger workgroups (8192 tokens, 4 sequences, 8 heads, us of `attend` and `attend_many`;
    // heads of 64: 64 rows 25 and 41, 128 rows 39 and 42, 256 rows 67 and 52; of 128: 32 rows 31 and 51, 64 rows 49 and 53, 128 rows 87 and 56;
    // of 256: 32 rows 61 and 82, 48 rows 88 and 84, 64 rows 114 and 86).
    p->many = p->rows * g.head_dim > 8192;
    p->qt = p->many || (p->rows > 16 && g.head_dim < 256) ? 2 : 1;       // (two groups of 16 rows of 256 do not fit the registers of `attend`)
    p->tile_rows = p->many ? 16 * p->qt * kWaves : 16 * p->qt;
    const uint64_t tiles = (p->rows + p->tile_rows - 1) / p->tile_rows;
    const uint64_t groups = tiles * g.seqs * g.heads;
    // steps that a row tile can have
    uint64_t tokens = g.table_blocks * g.block;
    if (g.window && g.window + p->tile_rows + 2 * kStep < tokens) tokens = g.window + p->tile_rows + 2 * kStep;
    const uint64_t steps = (tokens + kStep - 1) / kStep;
    // Parts of a tile: as many as make about eight workgroups a CU (two of the larger ones), which evens out sequences of different length, and no more than
    // its tokens can fill (part_of)
    const uint64_t want = p->many ? 512 : 2048;
    uint64_t splits = (want + groups - 1) / groups;
    const uint64_t most = (steps + kLeastPart - 1) / kLeastPart;
    splits = splits < most ? splits : most;
    if (p->many) {
        const uint64_t H = g.heads, ways = H % 8 == 0 ? 1 : 8 % H == 0 ? 8 / H : 8, per = H % 8 == 0 ? H / 8 : 8 % H == 0 ? 1 : H;
        const uint64_t positions = g.seqs * per * ((tiles + ways - 1) / ways);
        if (positions * 8 * splits >= uint64_t(1) << 24)
            return st_fail(ST_E_SHAPE, "%s: %llu workgroups are too many for one launch", kWho, (unsigned long long)(positions * 8 * splits));
        p->positions = uint32_t(positions);
    }
    if ((groups + 8 * tiles) * splits >= uint64_t(1) << 24)
        return st_fail(ST_E_SHAPE, "%s: %llu workgroups are too many for one launch", kWho, (unsigned long long)(groups * splits));
    p->tiles = uint32_t(tiles), p->splits = uint32_t(splits);
    if (splits > 1) {
        const uint64_t n = g.tokens * g.heads * g.group * splits;
        p->part_bytes = n * g.head_dim * 4, p->stat_bytes = n * sizeof(Part);
    }
    return ST_OK;
}

template <bool F16, int D>
void launch(const Args& a, const Plan& p, hipStream_t s) {
    const uint32_t heads = a.s.heads * a.s.seqs;
    if (p.many) hipLaunchKernelGGL((attend_many<F16, D, 2>), dim3(8 * p.positions * p.splits), dim3(kThreads), 0, s, a);
    else if (p.qt == 1) hipLaunchKernelGGL((attend<F16, D, 1>), dim3(p.tiles * heads * p.splits), dim3(kThreads), 0, s, a);
    else if constexpr (D < 256) hipLaunchKernelGGL((attend<F16, D, 2>), dim3(p.tiles * heads * p.splits), dim3(kThreads), 0, s, a);
    if (p.splits > 1) {
        constexpr uint32_t GROUPS = kThreads / (D / 4);
        uint32_t ways = 1;             // four parts or more for each
        while (ways < GROUPS && ways * 4 < p.splits) ways *= 2;
        const uint32_t per = GROUPS / ways;
        const uint64_t items = p.count * a.s.heads * a.group;
        hipLaunchKernelGGL((join<F16, D>), dim3(uint32_t((items + per - 1) / per), a.s.seqs), dim3(kThreads), 0, s, a, p.tile_rows, ways);
    }
}

}  // namespace

extern "C" st_status st_kv_attention_workspace_bytes(const st_kv_attention_args* g, uint64_t* bytes) {
    if (!bytes) return st_fail(ST_E_ARG, "st_kv_attention_workspace_bytes: null bytes");
    *bytes = 0;
    const st_status r = check_args(g);
    if (r != ST_OK || g->tokens == 0 || g->seqs == 0 || g->heads == 0 || g->group == 0) return r;
    Plan p;
    const st_status f = plan_of(*g, &p);
    if (f == ST_OK) *bytes = p.part_bytes + p.stat_bytes;
    return f;
}

extern "C" st_status st_kv_attention(const st_kv_attention_args* g, void* stream) {
    const st_status r = check_args(g);
    if (r != ST_OK || g->tokens == 0 || g->seqs == 0 || g->heads == 0 || g->group == 0) return r;
    Plan p;
    const st_status f = plan_of(*g, &p);
    if (f != ST_OK || p.rows == 0) return f;
    const uint64_t need = p.part_bytes + p.stat_bytes;
    if (need) {
        if (!g->workspace || g->workspace_bytes < need)
            return st_fail(ST_E_ARG, "%s: %llu bytes of workspace, %llu are needed", kWho,
                           (unsigned long long)(g->workspace ? g->workspace_bytes : 0), (unsigned long long)need);
        if (off(g->workspace, 16)) return st_fail(ST_E_ARG, "%s: workspace is not 16-byte aligned", kWho);
    }
    Args a = {};
    a.s = Seqs{g->table, g->lengths, g->starts, g->pages, g->table_blocks, g->table_pitch, uint32_t(g->tokens), uint32_t(g->seqs),
               uint32_t(g->max_new < g->tokens ? g->max_new : g->tokens), g->heads, stk::ilog2(g->block)};
    auto b = [](const void* v) { return static_cast<const uint8_t*>(v); };
    a.q = b(g->q); a.k = b(g->k); a.v = b(g->v); a.ks = b(g->k_scale); a.vs = b(g->v_scale);
    a.out = static_cast<uint8_t*>(g->out);
    if (need) {
        a.part = static_cast<float*>(g->workspace);
        a.stat = reinterpret_cast<Part*>(static_cast<uint8_t*>(g->workspace) + p.part_bytes);
    }
    a.q_pitch = g->q_pitch; a.q_head_pitch = g->q_head_pitch; a.out_pitch = g->out_pitch; a.out_head_pitch = g->out_head_pitch;
    a.group = g->group; a.causal = g->causal;
    a.window = uint32_t(g->window < (uint64_t(1) << 31) - 1 ? g->window : 0);      // as long as any sequence: all
    a.tiles = p.tiles; a.splits = p.splits;
    a.f = float(g->scale * 1.4426950408889634);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool h = g->q_type == ST_OUT_F16;
    if (g->head_dim == 64) h ? launch<true, 64>(a, p, s) : launch<false, 64>(a, p, s);
    else if (g->head_dim == 128) h ? launch<true, 128>(a, p, s) : launch<false, 128>(a, p, s);
    else h ? launch<true, 256>(a, p, s) : launch<false, 256>(a, p, s);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? ST_OK : st_fail(ST_E_HIP, "%s: launch failed: %s", kWho, hipGetErrorString(e));
}
