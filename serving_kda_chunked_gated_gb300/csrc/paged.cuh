// What the kernels over the paged key/value cache share: where a token lives, and the
// 8-bit rows.
#pragma once

#include <math.h>

#include "kda_common.cuh"

namespace kda {
namespace paged {

// a / b for 0 <= a, 0 < b; most quotients need no 64 bits
KDA_DEV long quotient(long a, long b) { return (a | b) >> 32 ? a / b : (long)((uint32_t)a / (uint32_t)b); }

// Sequences whose lens the kernels accept: the others are skipped.
KDA_DEV bool len_ok(const kda_paged_cache& c, int len) { return len >= 0 && len <= c.max_pages * c.page_size; }

// Where position `pos` of sequence n lies: a page table entry, as it was loaded, and the token in the page.  Apart from
// `row`, so that whoever looks ahead need not wait for the load.
struct Entry {
    int page, token;
};
KDA_DEV Entry entry_of(const kda_paged_cache& c, int n, int pos) {
    const int i = pos / c.page_size;
    return {c.tables[(size_t)n * c.max_pages + i], pos - i * c.page_size};
}
// Row of the flattened pages [num_pages page_size]; -1: a page outside the cache.
KDA_DEV int row(const kda_paged_cache& c, Entry e) {
    return (unsigned)e.page < (unsigned)c.num_pages ? e.page * c.page_size + e.token : -1;
}
KDA_DEV int row_of(const kda_paged_cache& c, int n, int pos) { return row(c, entry_of(c, n, pos)); }

// Sequence and position of packed row t; false: no sequence owns it, or one that is skipped.  cu NULL:
// one token of each sequence, or all of one.
struct Token {
    int n, pos;
};
KDA_DEV bool token_at(const kda_paged_cache& c, const int32_t* cu, int T, int t, Token* out) {
    int n = 0, end = T;
    if (cu) {
        if (t < cu[0] || t >= cu[c.num_seqs]) return false;
        int lo = 0, hi = c.num_seqs;                  // cu[lo] <= t < cu[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= t) lo = mid; else hi = mid;
        }
        n = lo;
        end = cu[n + 1];
    } else if (c.num_seqs > 1) {
        n = t;
        end = t + 1;
    }
    const int len = c.lens[n];
    if (!len_ok(c, len) || end <= t) return false;
    out->n = n;
    out->pos = len - (end - t);
    return true;
}

// ---------------------------------------------------------------------------
// 8-bit rows
// ---------------------------------------------------------------------------

// Exponent e of a row from the bits of its largest magnitude: the smallest with that at most
// 448 2^e = 1.75 2^(e + 8), from -100 to 119.  (Subnormal magnitudes end at -100 as well.)
KDA_DEV int row_exponent(uint32_t amax) {
    const int e = (int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u);
    return min(max(e, -100), 119);
}
KDA_DEV float power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }     // 2^e, -126 <= e <= 127

// what a scale byte stands for; 255: NaN
KDA_DEV float scale_of(uint32_t byte) { return __uint_as_float(byte == 255u ? 0x7fc00000u : byte << 23); }

// codes of (x0, x1), x0 in the low byte: nearest even, magnitudes past 448 to 448
KDA_DEV uint16_t codes2(float x0, float x1) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
    return r;
}
// the values of two codes in float32 (exact: fp16 holds every e4m3 number)
KDA_DEV float2 values2(uint16_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
    float2 v;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(v.x), "=f"(v.y) : "r"(h));
    return v;
}
// two codes as an fp16 pair (exact)
KDA_DEV uint32_t half2_of(uint32_t codes) {
    uint32_t h;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(codes));
    return h;
}
// a bf16 pair of the values times s (a power of two: exact), v.x lowest
KDA_DEV uint32_t scaled2(float2 v, float s) {
    uint32_t r;
    asm("{\n\t.reg .b64 v, s;\n\t.reg .f32 a, b;\n\tmov.b64 v, {%1, %2};\n\tmov.b64 s, {%3, %3};\n\t"
        "mul.rn.ftz.f32x2 v, v, s;\n\tmov.b64 {a, b}, v;\n\tcvt.rn.bf16x2.f32 %0, b, a;\n\t}" : "=r"(r) : "f"(v.x), "f"(v.y), "f"(s));
    return r;
}
// four codes as two bf16 pairs, times s, the first code lowest
KDA_DEV uint2 values4_bf16(uint32_t codes, float s) {
    return make_uint2(scaled2(values2((uint16_t)codes), s), scaled2(values2((uint16_t)(codes >> 16)), s));
}
// the larger magnitude of a bf16 pair, as float32 bits
KDA_DEV uint32_t magnitude(uint32_t w) { return max((w << 16) & 0x7fffffffu, w & 0x7fff0000u); }
}  // namespace paged
}  // namespace kda
