// A cache of keys and values in pages: its layout, and its 8-bit types.
#pragma once

#include "fs_attn_host.cuh"

namespace fs {
namespace kv {

using attn::View;

enum Held : int { HELD_16 = 0, HELD_E4M3 = 1, HELD_I8 = 2 };

constexpr float kTopE4m3 = 448.f, kTopI8 = 127.f;
constexpr float kLeastMax = 0x1p-80f;      // rows are scaled from this magnitude on
constexpr int kMaxTree = 256;              // tokens of a tree

// Rows of d elements of `bytes` bytes each; steps in bytes.
struct Pool {
    uint8_t* p;
    int64_t page, head, token;
    float* scale;                // scale of (page, head, token) at page * s_page + head * s_head + token
    int64_t s_page, s_head;
};

struct Cache {
    Pool k, v;
    const int32_t* table;
    int64_t table_stride;
    int table_pages;
    unsigned pages;
    int log_page;
    int G, d, held;
    int B;
    int vec16;                   // 8 bits: rows are whole aligned pieces of 16 bytes (else of 8)
    // page of position pos (>= 0) of sequence b, -1 without one
    __device__ __forceinline__ int page_of(int b, int pos) const {
        const int i = pos >> log_page;
        if (i >= table_pages) return -1;
        const int x = __ldg(table + b * table_stride + i);
        return (unsigned)x < pages ? x : -1;
    }
    __device__ __forceinline__ int slot_of(int pos) const { return pos & ((1 << log_page) - 1); }
    // positions that the table has
    __host__ __device__ __forceinline__ int reach() const { return table_pages << log_page; }
};

// Checks a description and fills `c`; `write`: its rows must not overlap.
fs_status fill_cache(int dev, Cache& c, const fs_cache* cache, bool write);

// The scales of a key and its value as a product's: the key's, and the value's logarithm.  A value
// scale that no row has (not positive, infinite, NaN, beyond 2^+-126) makes the key's scale NaN,
// and so every score with it: the rows that see the key are NaN, and the others never add
// what it comes to.
__device__ __forceinline__ bool weighable(float v_scale) { return v_scale >= 0x1p-126f && v_scale <= 0x1p126f; }
__device__ __forceinline__ void weigh(float k_scale, float v_scale, float& ks, float& lv) {
    const bool fine = weighable(v_scale);
    ks = fine ? k_scale : __uint_as_float(0x7fc00000u);
    lv = fine ? lg2(v_scale) : 0.f;
}

// Beside 8-bit values a row's reference is a whole number: value scales far apart bring it, and what it
// moves by, to 200, where float32 would round to 2^-17.
// x 2^y for a sum x of exponentials whose reference moves by -y; y may be below float32's exponents
// and x as much above 1: the factor goes in by halves.
__device__ __forceinline__ float moved_sum(float x, float y) {
    const float half = ex2(0.5f * y);
    return x * half * half;
}

// ref + log2(total), the exponent of total first: ref and it may be 120 and all but cancel.
__device__ __forceinline__ float log_sum(float ref, float total) {
    const int e = min(max((__float_as_int(total) >> 23) - 127, -126), 126);
    return (ref + (float)e) + lg2(total * __int_as_float((127 - e) << 23));
}

// Four codes as two registers of two float16 values each, in their order; exact.
template <int HELD>
__device__ __forceinline__ void widen4(uint32_t x, uint32_t& lo, uint32_t& hi) {
    if (HELD == HELD_E4M3) {
        asm("{\n\t.reg .b16 a, b;\n\t"
            "mov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(x));
    } else {
        // 128 more than the code in the low byte of 1024, less 1152
        x ^= 0x80808080u;
        const __half2 off = __half2half2(__ushort_as_half(0x6480));
        const uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
        const __half2 ha = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
        const __half2 hb = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
        lo = *reinterpret_cast<const uint32_t*>(&ha);
        hi = *reinterpret_cast<const uint32_t*>(&hb);
    }
}

}  // namespace kv
}  // namespace fs
