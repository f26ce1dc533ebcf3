// A cache of keys and values in pages: written from tokens, read back as tokens.
//
// Both are bound by memory alone: a row (one token of one key head, keys or values) is
// taken by 8 or 16 lanes, 16 bytes of 16-bit elements each, so that its largest
// magnitude is a few shuffles and nothing is read twice.
//
// Measured, 8 sequences of 4096 tokens, 8 heads of 128, bfloat16 to e4m3 and back: 78 us for both,
// 5.2 TB/s (0.77 of the measured copy rate); 5 x 777 float16 tokens of 4 heads of 80 to int8
// and 5 x 9001 back: 33 us, 2.7 TB/s (10 of a row's 16 lanes have elements, and many rows are
// zeros behind a sequence's end).
#include "fs_kv.cuh"

#include <cmath>

namespace fs {
namespace kv {

namespace {

using attn::check_ptr;

struct RowsArgs {
    Cache c;
    View k, v;               // tokens
    int n, bf16;
    const int32_t* at;       // write: positions; read: lengths, or nullptr
    int64_t at_stride;
    int vec;                 // token rows take 16-byte accesses
};

constexpr int kThreads = 256;
constexpr int kHeads = 4;       // heads of a token that a thread takes pieces of

template <typename T>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const T a = attn::from_f<T>(x), b = attn::from_f<T>(y);
    return (uint32_t)*reinterpret_cast<const uint16_t*>(&b) << 16 | *reinterpret_cast<const uint16_t*>(&a);
}
template <typename T>
__device__ __forceinline__ float elem(uint32_t w, int half) {
    const uint16_t u = (uint16_t)(half ? w >> 16 : w);
    return attn::to_f<T>(*reinterpret_cast<const T*>(&u));
}

__device__ __forceinline__ uint32_t word(const uint4& x, int k) {
    return k == 0 ? x.x : k == 1 ? x.y : k == 2 ? x.z : x.w;
}

template <typename T>
__device__ __forceinline__ constexpr uint32_t infinity_bits();
template <>
__device__ __forceinline__ constexpr uint32_t infinity_bits<__half>() { return 0x7c00u; }
template <>
__device__ __forceinline__ constexpr uint32_t infinity_bits<__nv_bfloat16>() { return 0x7f80u; }

// Elements 8 lane .. 8 lane + 7 of a token's row, zero from d on.
__device__ __forceinline__ uint4 load_piece(const uint16_t* row, int c, int d, bool vec) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (c >= d) return x;
    if (vec) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "l"(row + c));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = (uint32_t)row[c + 2 * k] | (uint32_t)row[c + 2 * k + 1] << 16;
        x = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return x;
}

// Largest magnitude of a row, in every one of its lanes, as 16 bits: those of a type's
// magnitudes are ordered as they are, infinities and NaN at the end.
template <int LANES>
__device__ __forceinline__ uint32_t row_top(const uint4& x) {
    uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                          __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    return max(m & 0xffffu, m >> 16);
}

// The 8-bit codes of a piece of a row that `up` brings to the type's range; not fine: zeros.
template <typename T, int HELD>
__device__ __forceinline__ uint2 codes(const uint4& x, float up, bool fine) {
    uint32_t w[2] = {0, 0};
    if (!fine) return make_uint2(0, 0);
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        const float a = __fmul_rn(elem<T>(word(x, k >> 1), 0), up), b = __fmul_rn(elem<T>(word(x, k >> 1), 1), up);
        uint32_t two;
        if (HELD == HELD_E4M3) {
            uint16_t h;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(b), "f"(a));
            two = h;
        } else {
            const int ia = min(max(__float2int_rn(a), -127), 127);
            const int ib = min(max(__float2int_rn(b), -127), 127);
            two = (uint32_t)(ia & 255) | (uint32_t)(ib & 255) << 8;
        }
        w[k >> 2] |= two << (8 * (k & 2));
    }
    return make_uint2(w[0], w[1]);
}

// A token's keys and values of up to kHeads heads to LANES lanes: one look at its page, and
// all their loads under way together.
struct Item {
    int b, t, h0, heads;       // heads 0: none
};
template <int LANES>
__device__ __forceinline__ Item item_of(const RowsArgs& P, unsigned items) {
    constexpr unsigned kItems = kThreads / LANES;
    const unsigned groups = (unsigned)(P.c.G + kHeads - 1) / kHeads;
    const unsigned i = blockIdx.x * kItems + threadIdx.x / LANES;
    const unsigned tok = i / groups, b = tok / (unsigned)P.n;
    const int h0 = (int)(i - tok * groups) * kHeads;
    return {(int)b, (int)(tok - b * (unsigned)P.n), h0, i < items ? min(kHeads, P.c.G - h0) : 0};
}

template <typename T, int HELD, int LANES>
__global__ void __launch_bounds__(kThreads) k_write(const __grid_constant__ RowsArgs P, unsigned items) {
    const Cache& c = P.c;
    const int lane = threadIdx.x % LANES;
    Item it = item_of<LANES>(P, items);
    int pos = -1, page = -1;
    if (it.heads > 0) pos = __ldg(P.at + it.b * P.at_stride + it.t);
    if (pos >= 0) page = c.page_of(it.b, pos);
    if (page < 0) it.heads = 0;
    const int slot = c.slot_of(pos);
    uint4 x[2 * kHeads];
#pragma unroll
    for (int i = 0; i < 2 * kHeads; ++i) {
        const View& from = i & 1 ? P.v : P.k;
        x[i] = make_uint4(0, 0, 0, 0);
        if (i >> 1 < it.heads)
            x[i] = load_piece(static_cast<const uint16_t*>(from.p) + it.b * from.sb + it.t * from.st +
                                  (it.h0 + (i >> 1)) * from.sh,
                              8 * lane, c.d, P.vec);
    }
    // The quotients of all rows, each by a lane of its own: top / amax by lane r (or 2 r) of row
    // r, amax / top by the same (or 2 r + 1), which writes it.  (Every lane dividing for every row
    // took a third of the kernel's instructions, and those its time.)
    static_assert(2 * kHeads == 8 && (LANES == 8 || LANES == 16), "lanes of the quotients");
    uint32_t top[2 * kHeads];
    float up = 0.f, scale = 0.f;
    if (HELD != HELD_16) {
        uint32_t mine = 0;
        const int r = LANES == 16 ? lane >> 1 : lane;
#pragma unroll
        for (int i = 0; i < 2 * kHeads; ++i) {
            top[i] = row_top<LANES>(x[i]);
            mine = i == r ? top[i] : mine;
        }
        constexpr float kTop = HELD == HELD_E4M3 ? kTopE4m3 : kTopI8;
        const float amax = fmaxf(elem<T>(mine, 0), kLeastMax);
        if (LANES == 16) {
            up = scale = __fdiv_rn(lane & 1 ? amax : kTop, lane & 1 ? kTop : amax);
        } else {
            up = __fdiv_rn(kTop, amax);
            scale = __fdiv_rn(amax, kTop);
        }
        const int h = it.h0 + (r >> 1);
        const Pool& to = r & 1 ? c.v : c.k;
        if ((LANES == 8 || lane & 1) && r >> 1 < it.heads)
            to.scale[page * to.s_page + h * to.s_head + slot] =
                mine < infinity_bits<T>() ? scale : __uint_as_float(0x7fc00000u);
    }
#pragma unroll
    for (int i = 0; i < 2 * kHeads; ++i) {
        const Pool& to = i & 1 ? c.v : c.k;
        const int h = it.h0 + (i >> 1);
        const bool on = i >> 1 < it.heads && 8 * lane < c.d;
        uint8_t* row = to.p + page * to.page + h * to.head + slot * to.token;
        if (HELD == HELD_16) {
            if (on) *reinterpret_cast<uint4*>(row + 16 * lane) = x[i];
        } else {
            const float by = __shfl_sync(0xffffffffu, up, LANES == 16 ? 2 * i : i, LANES);
            const uint2 q = codes<T, HELD>(x[i], by, top[i] < infinity_bits<T>());
            if (on) *reinterpret_cast<uint2*>(row + 8 * lane) = q;
        }
    }
}

template <typename T, int HELD>
__device__ __forceinline__ uint4 values(const uint2& q, float scale) {
    uint32_t w[4];
    widen4<HELD>(q.x, w[0], w[1]);
    widen4<HELD>(q.y, w[2], w[3]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        w[k] = pack2<T>(elem<__half>(w[k], 0) * scale, elem<__half>(w[k], 1) * scale);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int HELD, int LANES>
__global__ void __launch_bounds__(kThreads) k_read(const __grid_constant__ RowsArgs P, unsigned items) {
    const Cache& c = P.c;
    const int lane = threadIdx.x % LANES;
    const Item it = item_of<LANES>(P, items);
    if (it.heads == 0 || 8 * lane >= c.d) return;
    const int page = P.at == nullptr || it.t < __ldg(P.at + it.b) ? c.page_of(it.b, it.t) : -1;
    const int slot = c.slot_of(it.t);
    uint4 y[2 * kHeads];
    float scale[2 * kHeads];
#pragma unroll
    for (int i = 0; i < 2 * kHeads; ++i) {
        const Pool& from = i & 1 ? c.v : c.k;
        const int h = it.h0 + (i >> 1);
        y[i] = make_uint4(0, 0, 0, 0);
        scale[i] = 0.f;
        if (page < 0 || i >> 1 >= it.heads) continue;
        const uint8_t* row = from.p + page * from.page + h * from.head + slot * from.token;
        if (HELD == HELD_16) {
            y[i] = __ldg(reinterpret_cast<const uint4*>(row) + lane);
        } else {
            const uint2 q = __ldg(reinterpret_cast<const uint2*>(row) + lane);
            y[i].x = q.x;
            y[i].y = q.y;
            scale[i] = __ldg(from.scale + page * from.s_page + h * from.s_head + slot);
        }
    }
#pragma unroll
    for (int i = 0; i < 2 * kHeads; ++i) {
        if (i >> 1 >= it.heads) continue;
        const View& to = i & 1 ? P.v : P.k;
        // (a row without a page: zero codes by a zero scale)
        const uint4 o = HELD == HELD_16 ? y[i] : values<T, HELD>(make_uint2(y[i].x, y[i].y), scale[i]);
        uint16_t* out = static_cast<uint16_t*>(to.p) + it.b * to.sb + it.t * to.st + (it.h0 + (i >> 1)) * to.sh +
                        8 * lane;
        if (P.vec) {
            *reinterpret_cast<uint4*>(out) = o;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) out[k] = (uint16_t)(word(o, k >> 1) >> (16 * (k & 1)));
        }
    }
}

template <typename T, int HELD, int LANES>
cudaError_t launch(const RowsArgs& p, bool write, cudaStream_t s) {
    const int64_t items = (int64_t)p.c.B * p.n * ((p.c.G + kHeads - 1) / kHeads);     // below 2^31
    const unsigned grid = (unsigned)((items * LANES + kThreads - 1) / kThreads);
    if (write)
        k_write<T, HELD, LANES><<<grid, kThreads, 0, s>>>(p, (unsigned)items);
    else
        k_read<T, HELD, LANES><<<grid, kThreads, 0, s>>>(p, (unsigned)items);
    count_launch();
    return cudaGetLastError();
}
template <typename T, int HELD>
cudaError_t launch_lanes(const RowsArgs& p, bool write, cudaStream_t s) {
    return p.c.d <= 64 ? launch<T, HELD, 8>(p, write, s) : launch<T, HELD, 16>(p, write, s);
}
template <typename T>
cudaError_t launch_rows(const RowsArgs& p, bool write, cudaStream_t s) {
    if (p.c.held == HELD_16) return launch_lanes<T, HELD_16>(p, write, s);
    return p.c.held == HELD_E4M3 ? launch_lanes<T, HELD_E4M3>(p, write, s)
                                 : launch_lanes<T, HELD_I8>(p, write, s);
}

bool step_ok(const int64_t* s, int64_t pages, int heads, int tokens, int unit) {
    return (pages <= 1 || s[0] % unit == 0) && (heads <= 1 || s[1] % unit == 0) &&
           (tokens <= 1 || s[2] % unit == 0);
}

fs_status fill_pool(int dev, Pool& w, void* p, const int64_t* s, float* scale, const int64_t* ss,
                    const fs_cache* c, bool write, const char* name) {
    const int bytes = c->dtype >= FS_DTYPE_E4M3 ? 1 : 2;
    // strides in the order of a view: page, token, head
    const int64_t order[3] = {s[0], s[2], s[1]};
    View v;
    FS_TRY(attn::view(dev, v, p, order, c->pages, c->page_size, c->kv_heads, c->d, write, name));
    if (reinterpret_cast<uintptr_t>(p) % (8 * bytes) || !step_ok(s, c->pages, c->kv_heads, c->page_size, 8))
        return fail(FS_ERR_INVALID_ARG, "the rows of %s must start at multiples of %d bytes", name,
                    8 * bytes);
    w.p = static_cast<uint8_t*>(p);
    w.page = s[0] * bytes;
    w.head = s[1] * bytes;
    w.token = s[2] * bytes;
    w.scale = nullptr;
    w.s_page = w.s_head = 0;
    if (bytes == 1) {
        const int64_t so[3] = {ss[0], 1, ss[1]};
        FS_TRY(attn::view(dev, v, scale, so, c->pages, c->page_size, c->kv_heads, 1, write, "the scales"));
        w.scale = scale;
        w.s_page = ss[0];
        w.s_head = ss[1];
    }
    return FS_OK;
}

fs_status rows_entry(const fs_cache* cache, const fs_cache_rows* rows, const void* k, const void* v,
                     void* stream, bool write) {
    const int dev = attn::current_device();
    RowsArgs p = {};
    FS_TRY(fill_cache(dev, p.c, cache, write));
    if (!rows) return fail(FS_ERR_INVALID_ARG, "null fs_cache_rows");
    if (rows->dtype != FS_DTYPE_BF16 && rows->dtype != FS_DTYPE_F16)
        return fail(FS_ERR_INVALID_ARG, "fs_cache_rows.dtype=%d", rows->dtype);
    if (cache->dtype < FS_DTYPE_E4M3 && rows->dtype != cache->dtype)
        return fail(FS_ERR_INVALID_ARG, "tokens of dtype %d for a cache of dtype %d", rows->dtype,
                    cache->dtype);
    if (rows->reserved) return fail(FS_ERR_INVALID_ARG, "fs_cache_rows.reserved must be zero");
    constexpr int64_t kMaxTokens = INT32_MAX - 4096;
    if (rows->n < 0 || rows->n > kMaxTokens)
        return fail(FS_ERR_INVALID_ARG, "n=%lld out of range [0, %lld]", (long long)rows->n,
                    (long long)kMaxTokens);
    p.n = (int)rows->n;
    p.bf16 = rows->dtype == FS_DTYPE_BF16;
    const int64_t tokens = cache->batch * rows->n;
    FS_TRY(attn::view(dev, p.k, k, rows->k_stride, cache->batch, rows->n, p.c.G, p.c.d, !write, "k"));
    FS_TRY(attn::view(dev, p.v, v, rows->v_stride, cache->batch, rows->n, p.c.G, p.c.d, !write, "v"));
    if (write || rows->at) FS_TRY(check_ptr(dev, rows->at, tokens, write ? "positions" : "lengths"));
    if (write && rows->at_stride < 0) return fail(FS_ERR_INVALID_ARG, "negative at_stride");
    p.at = rows->at;
    p.at_stride = rows->at_stride;
    if ((double)tokens * p.c.G > (double)INT32_MAX)
        return fail(FS_ERR_UNSUPPORTED, "%.3g rows in one call", (double)tokens * p.c.G);
    if (tokens == 0) return FS_OK;
    p.vec = attn::aligned16(p.k, p.c.B, p.n, p.c.G) && attn::aligned16(p.v, p.c.B, p.n, p.c.G);
    NvtxRange range(write ? "fs_cache_write" : "fs_cache_read");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    FS_CUDA(p.bf16 ? launch_rows<__nv_bfloat16>(p, write, s) : launch_rows<__half>(p, write, s));
    return FS_OK;
}

}  // namespace

fs_status fill_cache(int dev, Cache& c, const fs_cache* a, bool write) {
    if (!a) return fail(FS_ERR_INVALID_ARG, "null fs_cache");
    if (a->dtype < FS_DTYPE_BF16 || a->dtype > FS_DTYPE_I8)
        return fail(FS_ERR_INVALID_ARG, "fs_cache.dtype=%d", a->dtype);
    constexpr int kMostHeads = 1 << 16;
    if (a->kv_heads < 1 || a->kv_heads > kMostHeads)
        return fail(FS_ERR_INVALID_ARG, "kv_heads=%d out of range [1, %d]", a->kv_heads, kMostHeads);
    if (a->d < 8 || a->d > attn::kMaxHeadDim || a->d % 8)
        return fail(FS_ERR_INVALID_ARG, "d=%d is not a multiple of 8 in [8, %d]", a->d, attn::kMaxHeadDim);
    if (a->page_size < 8 || a->page_size > 1 << 20 || (a->page_size & (a->page_size - 1)))
        return fail(FS_ERR_INVALID_ARG, "page_size=%d is not a power of two in [8, 2^20]", a->page_size);
    constexpr int64_t kMost = INT32_MAX - 4096;
    if (a->pages < 0 || a->pages > INT32_MAX || a->batch < 0 || a->batch > kMost || a->table_pages < 0 ||
        a->table_pages > kMost / a->page_size || a->table_stride < 0)
        return fail(FS_ERR_INVALID_ARG, "pages=%lld batch=%lld table_pages=%lld table_stride=%lld out of range",
                    (long long)a->pages, (long long)a->batch, (long long)a->table_pages,
                    (long long)a->table_stride);
    FS_TRY(fill_pool(dev, c.k, a->k, a->k_stride, a->k_scale, a->k_scale_stride, a, write, "cache.k"));
    FS_TRY(fill_pool(dev, c.v, a->v, a->v_stride, a->v_scale, a->v_scale_stride, a, write, "cache.v"));
    FS_TRY(check_ptr(dev, a->table, a->batch * a->table_pages, "the page table"));
    c.table = a->table;
    c.table_stride = a->table_stride;
    c.table_pages = a->pages ? (int)a->table_pages : 0;        // (no page: no position has one)
    c.pages = (unsigned)a->pages;
    c.log_page = 0;
    while (1 << c.log_page < a->page_size) ++c.log_page;
    c.G = a->kv_heads;
    c.d = a->d;
    c.held = a->dtype == FS_DTYPE_E4M3 ? HELD_E4M3 : a->dtype == FS_DTYPE_I8 ? HELD_I8 : HELD_16;
    c.B = (int)a->batch;
    const uintptr_t both = reinterpret_cast<uintptr_t>(a->k) | reinterpret_cast<uintptr_t>(a->v);
    c.vec16 = a->d % 16 == 0 && both % 16 == 0 && step_ok(a->k_stride, a->pages, c.G, a->page_size, 16) &&
              step_ok(a->v_stride, a->pages, c.G, a->page_size, 16);
    return FS_OK;
}

}  // namespace kv
}  // namespace fs

using namespace fs;

extern "C" {

fs_status fs_cache_write(const fs_cache* cache, const fs_cache_rows* rows, const void* k,
                         const void* v, void* stream) {
    try {
        return kv::rows_entry(cache, rows, k, v, stream, true);
    } catch (...) {
        return fail(FS_ERR_CUDA, "unexpected host exception");
    }
}

fs_status fs_cache_read(const fs_cache* cache, const fs_cache_rows* rows, void* k, void* v,
                        void* stream) {
    try {
        return kv::rows_entry(cache, rows, k, v, stream, false);
    } catch (...) {
        return fail(FS_ERR_CUDA, "unexpected host exception");
    }
}

}  // extern "C"
