// What the kernels that write (kv_append.hip) and read (attention.hip) the 8-bit cache share.
#pragma once

#include "matrix_codes.h"

namespace st_kv {

using namespace st_dev;

// New tokens of a sequence: rows first .. first + count - 1, at positions pos .. pos + count - 1 (pos may be negative), and the
// tokens that its table has room for.
struct Span {
    uint32_t first;
    int32_t count, pos, len;
};
struct Seqs {
    const int32_t *table, *lengths, *starts;
    uint64_t pages, table_blocks, table_pitch;
    uint32_t tokens, seqs, max_new;
    uint32_t heads, block_log2;
};

// Whatever the device arrays hold, rows stay below s.tokens and positions within the table.
__device__ __forceinline__ Span span_of(const Seqs& s, uint32_t seq) {
    Span p;
    int64_t a, b;
    if (s.starts) {
        a = s.starts[seq], b = s.starts[seq + 1];
        a = a < 0 ? 0 : a > s.tokens ? s.tokens : a;
        b = b < a ? a : b > s.tokens ? s.tokens : b;
    } else {
        const uint32_t per = s.tokens / s.seqs;
        a = uint64_t(seq) * per, b = a + per;
    }
    p.first = uint32_t(a);
    p.count = int32_t(b - a > s.max_new ? s.max_new : b - a);
    const int64_t room = int64_t(s.table_blocks) << s.block_log2, len = s.lengths[seq] < 0 ? 0 : s.lengths[seq];
    p.pos = int32_t(len - (b - a));
    p.len = int32_t(len > room ? room : len);
    return p;
}
// The page of block `at` of a sequence, or -1.
__device__ __forceinline__ int32_t page_of(const Seqs& s, uint32_t seq, int64_t at) {
    if (at < 0 || at >= int64_t(s.table_blocks)) return -1;
    const int32_t p = s.table[uint64_t(seq) * s.table_pitch + uint64_t(at)];
    return p >= 0 && uint64_t(p) < s.pages ? p : -1;
}
// The fp32 an E8M0 code stands for.
__device__ __forceinline__ float power_of(uint32_t code) {
    return code == 0 ? as_f32(0x00400000u) : code == 255 ? as_f32(0x7FC00000u) : as_f32(code << 23);
}

}  // namespace st_kv
