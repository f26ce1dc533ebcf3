// Cross attention, gradients, on the tensor cores.  The results are sums over
// different axes and no float atomics order them (results are bitwise repeatable), so
// the scores are formed for both: seven products where five are needed.
//
// grad_queries: a block takes 128 queries of one head and streams the keys.
//     S = Q K^T, dP = dO V^T, p = 2^{x - lse2}, ds = p (dP - delta),
//     dQ += ds K;   Q, dO and ds are A operands in TMEM.
//   Also the sums of ds by relative position for the bias gradient.
// grad_keys: a block takes 128 keys of one key head and streams the queries of
//   all its heads, with keys as rows:
//     S = K Q^T - lse2 / scale2, dP = V dO^T - delta, p = 2^{scale2 S},
//     dV += p dO, dK += p dP Q;   p and ds in TMEM.
//   There a row value belongs to a column, and reading 128 of each kind for every
//   thread took as long as the exponentials: they enter as one more product of 16 elements
//   (ones by three bfloat16 terms of each, 24 bits).
// Both run in one launch, after k_grad_rows (delta = dO . O) or k_grad_delta.  Where few
// blocks have many tiles, shares of them go to blocks of their own and k_grad_join adds
// the float32 sums in order.
//
// In both, eight warps hold the elementwise part (warps w and w + 4 the same 32
// rows, 64 columns of a tile each), and one thread issues the products in an order
// that keeps the tensor core at other products while a tile is in registers: p
// replaces S and ds replaces dP in TMEM as operands.  (Columns of their own for p
// and ds, as in the forward kernel, leave room for tiles of 64 only with wide heads:
// at batch 4, 2048 x 2048, 16 heads the gradients then took 374 instead of 341 us
// with heads of 64, 550 instead of 446 us with heads of 128.)  grad_queries has
// barriers and products for each half of a tile, so its two groups of four warps run out
// of step and one's latency is the other's work (heads of 128: 387 us for 407); in
// grad_keys products half as wide read shared memory half again as much, and lost.
//
// p and ds are rounded to the operands' 16 bits, sums are float32: in bfloat16 dq, dk and
// dv are 0.25 % off in the 2-norm, of which 0.17 % is their own rounding.  In float16 both
// are multiplied by powers of two first (kGradShift, range_shift), which the results' last
// factors take back: ds goes with dO, whose size is the training's choice, and as it is would
// be subnormal (dq and dk 0.8 % off at |dO| = 1e-4, 1500 keys) or infinite.  With the
// bounds on ds that takes 1 to 6 % of the gradients' time.
//
// Measured: batch 4, 2048 x 2048, 16 heads, bfloat16: 264 us with heads of 64 (650
// TFLOP/s of the five products; the chain of waits, exponentials and conversions of a
// tile, 2000 cycles for 1100 of products), 370 us with heads of 128 (930 TFLOP/s of the
// five, 1300 of the seven, 0.69 of the measured burst rate); in float16 4 to 5 % longer.
#include "fs_attn_host.cuh"

#include <atomic>
#include <type_traits>

namespace fs {
namespace attn {

namespace {

constexpr int kElemWarps = 8;
constexpr int kLoad = kElemWarps, kIssue = kElemWarps + 1, kClean = kElemWarps + 2;   // and one idle
constexpr int kGradThreads = 32 * (kElemWarps + 4);
constexpr int kSlack = 2 * kTile;
constexpr int kMaxRing = 8;
constexpr int kBands = 4;           // rows of bias sums: one per 32 queries

constexpr int kOnesBytes = 384 * kTile / 8;

struct GradBars {
    uint64_t full[kMaxRing], empty[kMaxRing], clean[kMaxRing];
    uint64_t own, ready, dvdone, done, drain;
    uint64_t sfull[2], sfree[2], dpfull[2], pfull, dsfull[2];    // grad_queries: of each half of a tile's keys
    uint32_t tmem, pad;
};

template <bool BF>
using Elem = typename std::conditional<BF, __nv_bfloat16, __half>::type;

// Two 16-bit values of a register as floats
template <bool BF>
__device__ __forceinline__ float2 unpack16(uint32_t u) {
    if (BF) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    const __half2 h = *reinterpret_cast<__half2*>(&u);
    return __half22float2(h);
}

// The half of a row of dsteps x 16 sums in TMEM, times `mul` (zero where !keep), rounded
// into a staged tile.  Whole warps.
template <int HD, bool BF>
__device__ __forceinline__ void stage_row(uint8_t* tile, int r, uint32_t tmem_row, int half, int dsteps,
                                          float mul, bool any, bool keep) {
    const int mid = (dsteps + 1) / 2 * 16;
    const int c0 = half ? mid : 0, c1 = half ? dsteps * 16 : mid;
    float o[HD / 2];
    if (any) {
#pragma unroll
        for (int c = 0; c < HD / 2; c += 32) tmem_ld32(tmem_row + c0 + c, o + c);
        tmem_wait_ld();
        tmem_reg_fence(o);
    }
#pragma unroll
    for (int c = 0; c < HD / 2; ++c) o[c] = any && keep ? o[c] * mul : 0.f;
#pragma unroll
    for (int c = 0; c < HD / 2; c += 16)
        if (c0 + c < c1) stage16<BF>(tile, r, c0 + c, o + c);
}

// The same, unrounded, to a row in memory: one share of the sum.
template <int HD>
__device__ __forceinline__ void part_row(float* out, bool live, uint32_t tmem_row, int half, int dsteps,
                                         float mul, bool any, int d) {
    const int mid = (dsteps + 1) / 2 * 16;
    const int c0 = half ? mid : 0, c1 = half ? d : min(mid, d);
    float o[HD / 2];
    if (any) {
#pragma unroll
        for (int c = 0; c < HD / 2; c += 32) tmem_ld32(tmem_row + c0 + c, o + c);
        tmem_wait_ld();
        tmem_reg_fence(o);
    }
#pragma unroll
    for (int c = 0; c < HD / 2; ++c)
        if (live && c0 + c < c1) out[c0 + c] = any ? o[c] * mul : 0.f;
    __syncwarp();
}

// base-2 bias of head h by relative position -D - kSlack .. D + kSlack
template <bool BF>
__device__ __forceinline__ void fill_bias(const Args& a, int h, float* sBias, int t, int threads) {
    const Elem<BF>* row = static_cast<const Elem<BF>*>(a.table) + h * a.table_stride;
#pragma unroll 4      // two loads that depend on one another an entry
    for (int e = t; e < 2 * (a.D + kSlack) + 1; e += threads)
        sBias[e] = bias2(to_f<Elem<BF>>(row[bucket_of(a, (int64_t)e - a.D - kSlack)]));
}

// ---------------------------------------------------------------------------

// Sums of a 32 x 32 block (a row per lane) along its diagonals, column - row = lane
// (upper) and lane - 32 (lower), through shared memory, ROWS rows of 33 floats at a
// time: in step s lane l reads column (s + l) mod 32 of row s.
template <int ROWS>
__device__ __forceinline__ void diagonals(const float* v, float* scratch, int lane, float& upper,
                                          float& lower) {
#pragma unroll 1
    for (int s0 = 0; s0 < 32; s0 += ROWS) {
        if (ROWS == 32 || lane / ROWS == s0 / ROWS) {
#pragma unroll
            for (int c = 0; c < 32; ++c) scratch[(lane - s0) * 33 + c] = v[c];
        }
        __syncwarp();
#pragma unroll 1
        for (int t = 0; t < ROWS; t += 8) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int c = s0 + t + u + lane;
                const float x = scratch[(t + u) * 33 + (c & 31)];
                if (c < 32)
                    upper += x;
                else
                    lower += x;
            }
        }
        __syncwarp();
    }
}

// grad_keys divides lse2 by scale2, which must not overflow: its scale2 is 2^-96 where it
// is less (the scores' share of x is below 2^-32 then), and a quotient stays within
// 2^120, where p = 0 for any finite bias that does not forbid its key.
constexpr float kRowLimit = 1.329227995784916e36f;      // 2^120
__device__ __forceinline__ float least_scale(const Args& a) { return fmaxf(a.scale2, 1.262177448353619e-29f); }

// x as three bfloat16 terms (24 bits), then five zeros
__device__ __forceinline__ uint4 three_terms(float x) {
    const float hi = __bfloat162float(__float2bfloat16_rn(x)), y = x - hi;
    const float mid = __bfloat162float(__float2bfloat16_rn(y));
    return make_uint4(pack16<true>(hi, mid), pack16<true>(y - mid, 0.f), 0u, 0u);
}

// -lse2 of a query; a row without a counted key has p = 0, as if its lse were +inf
__device__ __forceinline__ float row_lse(const Args& a, int b, int h, int64_t i) {
    const float x = i < a.n ? -a.lse[((int64_t)b * a.H + h) * a.n + i] * (float)kLog2e : -INFINITY;
    return x == INFINITY ? -INFINITY : x;
}
// row values of query r of its tile: x is -lse2, or -delta
__device__ __forceinline__ void put_row(const Args& a, uint8_t* out, int r, float x, bool is_delta) {
    reinterpret_cast<float*>(out + kRowBytes)[(is_delta ? kTile : 0) + r] = x;
    if (!is_delta) {
        x /= least_scale(a);
        if (x < -kRowLimit) x = -kRowLimit;
        if (x > kRowLimit) x = kRowLimit;
    }
    *reinterpret_cast<uint4*>(out + (r >> 3) * 256 + (is_delta ? 128 : 0) + (r & 7) * 16) = three_terms(x);
}

// float16: the power of two that ds is multiplied with, over whole tiles, so that a bound on it
// comes to [2^14, 2^15): the type then holds in full what is down to 2^-29 of that.  The
// bound is 2 max |dO_i| max |v_j| of the queries and values that meet, or, where
// k_grad_delta has formed all p dP, max |p_ij dP_ij| + |delta_i|.  Rows that are not finite
// set none: they are lost with any.  A whole warp.
__device__ __forceinline__ float range_max(const float* x, int count) {
    float top = 0.f;
#pragma unroll 4
    for (int e = threadIdx.x & 31; e < count; e += 32) top = fmaxf(top, __ldg(x + e));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top;
}
__device__ __forceinline__ int range_shift(const GradArgs& P, int b, int h, int tile, int tiles) {
    const Args& a = P.a;
    float bound = range_max(P.q_range + (((int64_t)b * a.H + h) * P.q_tiles + tile) * 4, 4 * tiles);
    if (!P.exact_delta)
        bound *= 2.f * range_max(P.v_range + ((int64_t)b * a.G + h / a.R) * P.k_tiles, P.k_tiles);
    return bound > 0.f ? min(14 + 127 - (int)(__float_as_uint(bound) >> 23), 100) : 0;
}
__device__ __forceinline__ float power2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ float finite_or_0(float x) { return x < INFINITY ? x : 0.f; }
// the entry of a warp's 32 queries of a tile
__device__ __forceinline__ void put_range(const GradArgs& P, int64_t tile, int quarter, int lane, float x) {
    x = finite_or_0(x);
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    if (lane == 0) P.q_range[tile * 4 + quarter] = x;
}

// p of grad_keys in float16 is multiplied by 2^kGradShift: in full down to 2^-28, and no more
// than the rounding of x can take it past 1 would make it infinite
constexpr int kGradShift = 14;

// ---------------------------------------------------------------------------
// The row values of 128 queries a block: delta_i = dO_i . O_i and lse_i.  Reads dO and O
// once, LANES lanes of 8 elements to a row; bound by memory (4 x 2048 x 16 rows of 128: 68 MB
// in 18 us from a cold cache).  In float16 also the norms of dO and, in blocks of their own
// behind those, of V.

constexpr int kRowThreads = 256;

// The row's elements [c, c + 8) as 4 registers, zero beyond d; `vec`: 16-byte loads
__device__ __forceinline__ void load8(const View& w, int64_t off, int c, int d, bool live, bool vec,
                                      uint32_t* u) {
    const uint16_t* p = static_cast<const uint16_t*>(w.p) + off;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (live && vec) {
        if (c < d) x = __ldg(reinterpret_cast<const uint4*>(p + c));
    } else if (live) {
        uint32_t* xs = &x.x;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c + k < d) xs[k >> 1] |= (uint32_t)__ldg(p + c + k) << (16 * (k & 1));
    }
    u[0] = x.x;
    u[1] = x.y;
    u[2] = x.z;
    u[3] = x.w;
}

// The largest norm of a counted value of a key tile
template <int LANES>
__device__ __forceinline__ void value_range(const GradArgs& P, int64_t blk) {
    constexpr int kRows = 32 / LANES, kTurns = 16 / kRows;
    __shared__ float sTop[kRowThreads / 32];
    const Args& a = P.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = (int)(blk % P.k_tiles), g = (int)(blk / P.k_tiles % a.G), b = (int)(blk / P.k_tiles / a.G);
    const uint4 w = tile_words(P.kt, b, tile, key_end(a, b));
    const uint32_t word = warp < 2 ? w.x : warp < 4 ? w.y : warp < 6 ? w.z : w.w;    // of the warp's 16 keys
    uint32_t u[kTurns][4];
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int r = warp * 16 + k * kRows + lane / LANES;
        // (V as the tensor map reads it: its rows take 16-byte loads)
        load8(a.v, b * a.v.sb + ((int64_t)tile * kTile + r) * a.v.st + g * a.v.sh, 8 * (lane % LANES), a.d,
              (word >> (r & 31)) & 1u, true, u[k]);
    }
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack16<false>(u[k][e]);
            x = fmaf(f.x, f.x, x);
            x = fmaf(f.y, f.y, x);
        }
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        top = fmaxf(top, finite_or_0(x));
    }
#pragma unroll
    for (int o = 16; o >= LANES; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) sTop[warp] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int k = 1; k < kRowThreads / 32; ++k) top = fmaxf(top, sTop[k]);
        P.v_range[blk] = sqrtf(top);
    }
}

template <int LANES, bool BF>
__global__ void __launch_bounds__(kRowThreads) k_grad_rows(const __grid_constant__ GradArgs P) {
    constexpr int kRows = 32 / LANES, kTurns = 16 / kRows;      // rows of a warp at a time, of 16
    __shared__ float sDelta[kTile], sNorm[BF ? 1 : kTile];
    const Args& a = P.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (!BF) {
        const int queries = P.q_tiles * a.H * a.B;
        if ((int)blockIdx.x >= queries) {
            value_range<LANES>(P, (int)blockIdx.x - queries);
            return;
        }
    }
    int blk = blockIdx.x;
    const int qt = blk % P.q_tiles;
    blk /= P.q_tiles;
    const int h = blk % a.H, b = blk / a.H;
    const int c = 8 * (lane % LANES);
    uint32_t u[kTurns][4], v[kTurns][4];
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int64_t i = qt * kTile + warp * 16 + k * kRows + lane / LANES;
        load8(a.dout, b * a.dout.sb + i * a.dout.st + h * a.dout.sh, c, a.d, i < a.n, P.dout_vec, u[k]);
        load8(a.o, b * a.o.sb + i * a.o.st + h * a.o.sh, c, a.d, i < a.n, P.o_vec, v[k]);
    }
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        float dot = 0.f, norm = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack16<BF>(u[k][e]), g = unpack16<BF>(v[k][e]);
            dot = fmaf(f.x, g.x, dot);
            dot = fmaf(f.y, g.y, dot);
            if (!BF) norm = fmaf(f.x, f.x, fmaf(f.y, f.y, norm));
        }
        const int r = warp * 16 + k * kRows + lane / LANES;
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) {
            dot += __shfl_xor_sync(0xffffffffu, dot, o);
            if (!BF) norm += __shfl_xor_sync(0xffffffffu, norm, o);
        }
        if (lane % LANES == 0) sDelta[r] = dot;
        if (!BF && lane % LANES == 0) sNorm[r] = norm;
    }
    __syncthreads();
    const int r = threadIdx.x & (kTile - 1);
    const bool second = threadIdx.x >= kTile;
    const int64_t tile = ((int64_t)b * a.H + h) * P.q_tiles + qt;
    put_row(a, P.rows + tile * kRowStride, r, second ? -sDelta[r] : row_lse(a, b, h, (int64_t)qt * kTile + r),
            second);
    if (!BF && !second) put_range(P, tile, warp, lane, sqrtf(sNorm[r]));
}

// ---------------------------------------------------------------------------

// Q and dO are copied to TMEM once (as A operands in shared memory they are read with
// every product: 94 instead of 67 us for 304 blocks of 16 key tiles, heads of 128,
// although TMEM then has room for two dP tiles).
template <int HD>
struct GradQ {
    static constexpr int kKeys = kTile, kCols = kTile / 2;       // keys of a tile, of a warp
    static constexpr int kChunks = HD / 64, kChunkBytes = CHUNK_BYTES;
    static constexpr int kTileBytes = kChunks * CHUNK_BYTES;
    static constexpr uint32_t S = 0, DP = kTile, DQ = DP + kTile, Q = DQ + HD, DO = Q + HD / 2;    // TMEM columns
    static_assert(DO + HD / 2 <= 512, "TMEM");
};

// DELTA: no gradients, only the row values, with delta_i = sum_j p_ij dP_ij in float32.
// With delta from the 16-bit O, sum_j ds_ij is dO_i . (error of O_i) instead of 0, and a
// bucket that holds nearly all of its rows' weight sums nothing but that: its gradient
// came out up to 1.2 % off (2-norm of dbias against 64 bits, 0.24 % with this pass).  It
// costs a quarter of the gradients' time, so only a bias gradient and calls with few keys
// take it (exact_delta).
template <int HD, bool BF, bool DELTA>
__device__ __forceinline__ void grad_queries(const GradArgs& P, int blk) {
    using C = GradQ<HD>;
    constexpr int KT = C::kKeys, NC = C::kCols;
    constexpr uint64_t kTileU = C::kTileBytes >> 4, kHalfU = (uint64_t)(NC * 128) >> 4;   // descriptor units
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    const Args& a = P.a;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int NS = DELTA ? P.delta_stages : P.stages;                // even: K and V keep their slots
    uint8_t* sKV = smem;                    // at first Q and dO in the last two tiles, at the end dq
    uint8_t* sOwn = sKV + (NS - 2) * C::kTileBytes;
    GradBars& bar = *reinterpret_cast<GradBars*>(sKV + NS * C::kTileBytes);
    float* sFar = reinterpret_cast<float*>(&bar + 1);            // [8][2], or the second halves' sums and largest
    float* sBias = sFar + (DELTA ? 2 * kTile : 2 * kElemWarps);      // [2 (D + kSlack) + 1]
    float* sSums = sBias + (a.table ? 2 * (a.D + kSlack) + 1 : 0);   // [4][2 D + 1]
    float* sScratch = sSums + kBands * (2 * a.D + 1);            // [8][scratch_rows][33], with bias sums

    const int split = blk % P.q_splits;
    blk /= P.q_splits;
    const int qt = blk % P.q_tiles;
    blk /= P.q_tiles;
    const int h = blk % a.H;
    const int b = longest_first<KT>(P.kt, a, blk / a.H);
    const int i0 = qt * kTile;
    const int end = key_end(a, b);
    const int nt_all = step_count<KT>(P.kt, b, end), per = (nt_all + P.q_splits - 1) / P.q_splits;
    const int t0 = min(nt_all, split * per), nt = min(nt_all, t0 + per) - t0;
    const bool partial_keys = !DELTA && (P.kt.words != nullptr || end < a.m);
    const int64_t first = (a.q_pos ? (int64_t)__ldg(a.q_pos + b) : 0) + i0;
    const int dsteps = (a.d + 15) >> 4, dchunks = (a.d + 63) >> 6;
    const int width = 2 * a.D + 1;

    if (warp == kLoad) {
        if (lane < NS) mbar_init(&bar.full[lane], 1);
        if (lane == NS) mbar_init(&bar.own, 1);
        if (lane == NS + 1) mbar_init(&bar.ready, kElemWarps);
        fence_mbar_init();
        __syncwarp();
    } else if (warp == kClean) {
        if (lane < NS) {
            mbar_init(&bar.empty[lane], 1);
            mbar_init(&bar.clean[lane], 1);
        } else if (lane == NS) {
            for (int u = 0; u < 2; ++u) {
                mbar_init(&bar.sfull[u], 1);
                mbar_init(&bar.sfree[u], kElemWarps / 2);
                mbar_init(&bar.dpfull[u], 1);
                mbar_init(&bar.dsfull[u], kElemWarps / 2);
            }
            mbar_init(&bar.done, 1);
            mbar_init(&bar.drain, 1);
        }
        fence_mbar_init();
    }
    if (warp == kIssue) tmem_alloc(&bar.tmem, 512);
    const auto load = [&](int it, int slot) {      // K and V tiles in turn
        const int g = h / a.R;
        const int key = step_key<KT>(P.kt, b, t0 + (it >> 1));
        const TensorMap& src = it & 1 ? P.v : P.k;
        mbar_arrive_expect_tx(&bar.full[slot], C::kTileBytes);
        for (int c = 0; c < C::kChunks; ++c)
            tma_load(sKV + slot * C::kTileBytes + c * C::kChunkBytes, &src.map, c * 64, key, g * src.head,
                     b * src.batch, &bar.full[slot]);
    };
    const int early = min(2 * nt, NS - 2);         // copies that need no free slot
    if (warp == kLoad && nt > 0 && elect_one()) {
        mbar_arrive_expect_tx(&bar.own, 2 * C::kTileBytes);
        for (int c = 0; c < C::kChunks; ++c) {
            tma_load(sOwn + c * CHUNK_BYTES, &P.q.map, c * 64, i0, h * P.q.head, b * P.q.batch, &bar.own);
            tma_load(sOwn + C::kTileBytes + c * CHUNK_BYTES, &P.dout.map, c * 64, i0, h * P.dout.head,
                     b * P.dout.batch, &bar.own);
        }
        for (int it = 0; it < early; ++it) load(it, it);
    }
    if (a.table) fill_bias<BF>(a, h, sBias, threadIdx.x, kGradThreads);
    if (!DELTA && a.bias_part)
        for (int e = threadIdx.x; e < kBands * width; e += kGradThreads) sSums[e] = 0.f;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;

    if (warp == kLoad) {
        if (nt > 0 && elect_one()) {
            Ring r;
            r.step(early, NS);
            int issued = early;
            bool ok = true;
            for (int it = early; it < 2 * nt; ++it) {
                // (Q and dO have left the last two slots before their first use)
                if (it == NS - 2) ok = mbar_wait(&bar.ready, 0, a.err, ERR_TIMEOUT_PRODUCER);
                ok = ok && mbar_wait(&bar.empty[r.slot], r.phase ^ 1u, a.err, ERR_TIMEOUT_PRODUCER);
                if (!ok) break;
                load(it, r.slot);
                ++issued;
                r.step(1, NS);
            }
            if (!ok) {   // every copy lands before the block can exit
                mbar_wait(&bar.own, 0, a.err, ERR_TIMEOUT_PRODUCER);
                Ring l;
                for (int it = 0; it < issued; ++it) {
                    if (it + NS >= issued)
                        mbar_wait(&bar.full[l.slot], l.phase, a.err, ERR_TIMEOUT_PRODUCER);
                    l.step(1, NS);
                }
            }
        }
    } else if (warp == kIssue) {
        if (nt > 0 && elect_one()) {
            const uint32_t idS = idesc_16(BF, NC, false);
            const uint32_t idQ = idesc_16(BF, dsteps * 16, true);
            const uint64_t dKV = sdesc_sw128(smem_u32(sKV)), dKVt = sdesc_tokens(smem_u32(sKV));
            uint64_t* kbar = partial_keys ? bar.clean : bar.full;
            Ring r;
            // scores of half u of the tile at r, and its dP from the V tile beside it
            const auto scores = [&](int u) {
                mma_over_d_ts(tmem + C::S + u * NC, tmem + C::Q, dKV + r.slot * kTileU + u * kHalfU,
                                           idS, dchunks);
                mma_commit(&bar.sfull[u]);
                if (DELTA && u) mma_commit(&bar.empty[r.slot]);
            };
            const auto grads = [&](int u) {
                mma_over_d_ts(tmem + C::DP + u * NC, tmem + C::DO,
                                           dKV + (r.slot + 1) * kTileU + u * kHalfU, idS, dchunks);
                mma_commit(&bar.dpfull[u]);
                if (u) mma_commit(&bar.empty[r.slot + 1]);
            };
            bool ok = mma_wait(a.err, &bar.ready, 0) && mma_wait(a.err, &kbar[0], 0) &&
                      mma_wait(a.err, &bar.full[1], 0);
            if (ok) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    scores(u);
                    grads(u);
                }
            }
            for (int j = 0; j < nt && ok; ++j) {
                const bool more = j + 1 < nt;
                const uint64_t dTile = dKVt + r.slot * kTileU;
                uint64_t* const done_with = &bar.empty[r.slot];
                r.step(2, NS);
                // (copies that have long landed are waited for before the warps)
                bool seen = false;
                if (more) {
                    const bool k_seen = mbar_test(&kbar[r.slot], r.phase);
                    const bool v_seen = mbar_test(&bar.full[r.slot + 1], r.phase);
                    seen = mbar_test(&bar.sfree[0], j & 1);
                    ok = (k_seen || mma_wait(a.err, &kbar[r.slot], r.phase)) &&
                         (v_seen || mma_wait(a.err, &bar.full[r.slot + 1], r.phase));
                    if (!ok) break;
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (more) {      // scores of the next tile, once this one's are in registers
                        if (!(ok = seen || mma_wait(a.err, &bar.sfree[u], j & 1))) break;
                        tc_fence_after();
                        scores(u);
                    }
                    const bool ds_seen = mbar_test(&bar.dsfull[u], j & 1);
                    seen = u == 0 && more && mbar_test(&bar.sfree[1], j & 1);
                    if (!(ok = ds_seen || mma_wait(a.err, &bar.dsfull[u], j & 1))) break;
                    tc_fence_after();
                    if (!DELTA) {
                        mma_over_tokens<NC>(tmem + C::DQ, tmem + C::DP + u * NC, dTile + u * kHalfU, idQ,
                                            j > 0 || u > 0, 0);
                        if (u) mma_commit(done_with);
                    }
                    if (more) grads(u);
                }
            }
            mma_commit(&bar.done);
            mma_commit(&bar.drain);
            mbar_wait(&bar.drain, 0, a.err, ERR_TIMEOUT_MMA);
        }
    } else if (warp == kClean) {
        if (partial_keys) {
            Ring r;
            for (int j = 0; j < nt; ++j) {
                const KeyBits<KT> w(P.kt, b, t0 + j, end);
                if (!warp_wait(&bar.full[r.slot], r.phase, a.err, ERR_TIMEOUT_PRODUCER)) break;
                if (!w.all()) {
                    clear_rows(sKV + r.slot * C::kTileBytes, C::kChunks, C::kChunkBytes, w, lane);
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.clean[r.slot]);
                r.step(2, NS);
            }
        }
    } else if (warp < kElemWarps) {
        const int quarter = warp & 3, half = warp >> 2;
        const int r = quarter * 32 + lane;
        const int i = i0 + r;
        const uint32_t lofs = (uint32_t)(quarter * 32) << 16;
        uint8_t* const values = P.rows + (((int64_t)b * a.H + h) * P.q_tiles + qt) * kRowStride;
        const float* row = reinterpret_cast<const float*>(values + kRowBytes);
        // float16: ds, and the sums of the bias gradient, are 2^shift times as large
        const int shift = BF || DELTA ? 0 : range_shift(P, b, h, qt, 1);
        float nlse = DELTA ? row_lse(a, b, h, i) : row[r];
        if (!BF && !DELTA) nlse += (float)shift;
        const float ndelta = DELTA ? 0.f : row[kTile + r];
        bool ok = true;
        if (nt > 0) {     // operands into TMEM: warps 0..3 the rows of Q, warps 4..7 those of dO
            ok = warp_wait(&bar.own, 0, a.err, ERR_TIMEOUT_EPILOGUE);
            const uint8_t* src = sOwn + half * C::kTileBytes;
#pragma unroll 4
            for (int x = 0; x < 4 * dchunks; ++x) {
                uint32_t u[8];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint4 y = *reinterpret_cast<const uint4*>(
                        src + (x >> 2) * CHUNK_BYTES + swz_offset(r, (x & 3) * 16 + 8 * e));
                    u[4 * e] = y.x;
                    u[4 * e + 1] = y.y;
                    u[4 * e + 2] = y.z;
                    u[4 * e + 3] = y.w;
                }
                tmem_st8u(tmem + lofs + (half ? C::DO : C::Q) + 8 * x, u);
            }
            tmem_wait_st();
            tc_fence_before();
            fence_proxy_async_smem();      // the slots are copied over next
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.ready);
        }
        const uint32_t tS = tmem + lofs + C::S + half * NC, tDP = tmem + lofs + C::DP + half * NC;
        float* scratch = sScratch + warp * P.scratch_rows * 33;
        float far_lo = 0.f, far_hi = 0.f, total = 0.f, top = 0.f;      // DELTA: sum, and largest, of p dP
        for (int j = 0; j < nt && ok; ++j) {
            // relative position of the warp's first row and column
            const int64_t rel0 =
                a.table ? step_key<KT>(P.kt, b, t0 + j) + half * NC - first - quarter * 32 : (int64_t)0;
            if (!(ok = warp_wait(&bar.sfull[half], j & 1, a.err, ERR_TIMEOUT_EPILOGUE))) break;
            tc_fence_after();
            float v[NC];
#pragma unroll
            for (int c = 0; c < NC; c += 32) tmem_ld32(tS + c, v + c);
            tmem_wait_ld();
            tmem_reg_fence(v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.sfree[half]);
            const bool dp_seen = mbar_test(&bar.dpfull[half], j & 1);
            float mul = a.scale2, add = 0.f;
            int where = 0;                       // -1, 1: every pair beyond -D or D
            if (a.table) {
                if (rel0 - 31 >= a.D) {
                    add = sBias[2 * a.D + kSlack];
                    where = 1;
                } else if (rel0 + (NC - 1) <= -a.D) {
                    add = sBias[kSlack];
                    where = -1;
                } else {
                    const float* e = sBias + (int)rel0 - lane + a.D + kSlack;
#pragma unroll
                    for (int c = 0; c < NC; ++c) v[c] = fmaf(v[c], mul, e[c]);
                    mul = 1.f;
                }
            }
            const float base = add + nlse;
            const uint64_t mul2 = pk(mul, mul), base2 = pk(base, base);
#pragma unroll
            for (int c = 0; c < NC; c += 2) {
                upk(fma2(pk(v[c], v[c + 1]), mul2, base2), v[c], v[c + 1]);
                v[c] = ex2(v[c]);
                v[c + 1] = ex2(v[c + 1]);
            }
            if (!(ok = __all_sync(0xffffffffu, dp_seen) ||
                       warp_wait(&bar.dpfull[half], j & 1, a.err, ERR_TIMEOUT_EPILOGUE)))
                break;
            tc_fence_after();
            {
                float g[NC];
#pragma unroll
                for (int c = 0; c < NC; c += 32) tmem_ld32(tDP + c, g + c);
                tmem_wait_ld();
                tmem_reg_fence(g);
                if (DELTA) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.dsfull[half]);
                }
                const uint64_t nd = pk(ndelta, ndelta);
#pragma unroll
                for (int c = 0; c < NC; c += 2)
                    upk(mul2f(pk(v[c], v[c + 1]), add2(pk(g[c], g[c + 1]), nd)), v[c], v[c + 1]);
            }
            if (P.kt.words || (t0 + j + 1) * KT > end) {
                const KeyBits<KT> w(P.kt, b, t0 + j, end);
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const uint32_t bits = half ? w.w[2 + (c >> 5)] : w.w[c >> 5];
                    if (!((bits >> (c & 31)) & 1u)) v[c] = 0.f;
                }
            }
            if (DELTA) {
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int c = 0; c < NC; c += 2) {
                    s0 += v[c];
                    s1 += v[c + 1];
                    if (!BF) top = max3(top, fabsf(v[c]), fabsf(v[c + 1]));
                }
                total += s0 + s1;
            } else {
                uint32_t u[NC / 2];
#pragma unroll
                for (int c = 0; c < NC / 2; ++c) u[c] = pack16<BF>(v[2 * c], v[2 * c + 1]);
                tmem_st32(tDP, u);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.dsfull[half]);
            }
            if (!DELTA && a.bias_part) {
                if (where != 0) {
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int c = 0; c < NC; c += 2) {
                        s0 += v[c];
                        s1 += v[c + 1];
                    }
                    if (where > 0)
                        far_hi += s0 + s1;
                    else
                        far_lo += s0 + s1;
                } else {
                    // upper[q] and lower[q] of lane l are at relative position rel0 + 32 q + l and
                    // 32 less.  A diagonal of these 32 rows meets two 32 x 32 blocks at most, so no
                    // entry of the sums gets more than two terms, and the order of the two
                    // additions between warps does not matter.
                    float* sums = sSums + quarter * width + a.D;
                    const auto put = [&](int rel, float x, bool alone) {
                        if (rel >= a.D)
                            far_hi += x;
                        else if (rel <= -a.D)
                            far_lo += x;
                        else if (alone)
                            sums[rel] = x;
                        else
                            atomicAdd(sums + rel, x);
                    };
                    float upper[NC / 32], lower[NC / 32];
#pragma unroll
                    for (int q = 0; q < NC / 32; ++q) {
                        upper[q] = lower[q] = 0.f;
                        if (P.scratch_rows == 32)
                            diagonals<32>(v + 32 * q, scratch, lane, upper[q], lower[q]);
                        else if (P.scratch_rows == 16)
                            diagonals<16>(v + 32 * q, scratch, lane, upper[q], lower[q]);
                        else
                            diagonals<8>(v + 32 * q, scratch, lane, upper[q], lower[q]);
                    }
                    static_assert(NC == 64, "two blocks a warp");
                    const int rel = (int)rel0 + lane;
                    if (lane > 0) put(rel - 32, lower[0], false);
                    put(rel, upper[0] + lower[1], true);
                    put(rel + 32, upper[1], lane == 0);
                }
            }
        }
        if (DELTA) {       // the two halves of a row, to its row values
            if (half) {
                sFar[r] = total;
                if (!BF) sFar[kTile + r] = top;
            }
            named_sync(2 + quarter, 64);
            total += sFar[r];
            if (!BF) top = fmaxf(top, sFar[kTile + r]);
            const int64_t tile = ((int64_t)b * a.H + h) * P.q_tiles + qt;
            if (P.q_splits > 1) {
                const int64_t at = ((int64_t)split * a.B * a.H * P.q_tiles + tile) * kTile + r;
                if (ok && !half) {
                    P.part_delta[at] = total;
                    if (!BF) P.part_top[at] = top;
                }
            } else if (ok) {
                put_row(a, values, r, half ? nlse : -total, !half);
                if (!BF && !half) put_range(P, tile, quarter, lane, top + fabsf(total));
            }
        }
        if (!DELTA && nt > 0 && ok) ok = warp_wait(&bar.done, 0, a.err, ERR_TIMEOUT_EPILOGUE);
        tc_fence_after();
        const bool whole = P.q_splits == 1;
        const float scale = BF ? a.scale : a.scale * power2(-shift);
        if (!DELTA && ok) {
            if (whole)
                stage_row<HD, BF>(sKV, r, tmem + lofs + C::DQ, half, dsteps, scale, nt > 0, true);
            else
                part_row<HD>(P.part_dq + (((int64_t)split * a.B + b) * a.H + h) * a.n * a.d + (int64_t)i * a.d,
                             i < a.n, tmem + lofs + C::DQ, half, dsteps, scale, nt > 0, a.d);
        }
        named_sync(2 + quarter, 64);
        if (!DELTA && ok && whole) {
            const int w0 = i - lane + half * 16;
            unstage_rows<16>(sKV, quarter * 32 + half * 16, a.n - w0, a.d,
                             static_cast<uint16_t*>(a.dq.p) + b * a.dq.sb + (int64_t)w0 * a.dq.st + h * a.dq.sh,
                             a.dq.st, P.dq_vec, lane);
        }
        if (!DELTA && a.bias_part) {
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                far_lo += __shfl_xor_sync(0xffffffffu, far_lo, o);
                far_hi += __shfl_xor_sync(0xffffffffu, far_hi, o);
            }
            if (lane == 0) {
                sFar[2 * warp] = far_lo;
                sFar[2 * warp + 1] = far_hi;
            }
            named_sync(1, 32 * kElemWarps);
            float* out = a.bias_part + ((((int64_t)h * a.B + b) * P.q_tiles + qt) * P.q_splits + split) * width;
            for (int e = threadIdx.x; e < width; e += 32 * kElemWarps) {
                float s = 0.f;
                if (e == 0 || e == width - 1) {
#pragma unroll
                    for (int k = 0; k < kElemWarps; ++k) s += sFar[2 * k + (e ? 1 : 0)];
                } else {
#pragma unroll
                    for (int k = 0; k < kBands; ++k) s += sSums[k * width + e];
                }
                out[e] = BF ? s : s * power2(-shift);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kIssue) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------

template <int HD>
struct GradKV {
    static constexpr int kQueries = kTile, kCols = kTile / 2;    // queries of a tile, of a warp
    static constexpr int kChunks = HD / 64, kChunkBytes = CHUNK_BYTES;
    static constexpr int kTileBytes = kChunks * CHUNK_BYTES;
    static constexpr int kOwnBytes = kTileBytes;                 // the block's K or V
    static constexpr uint32_t S = 0, DP = kTile, DV = 2 * kTile, DK = 3 * kTile;     // TMEM columns
};

template <int HD, bool BF>
__device__ __forceinline__ void grad_keys(const GradArgs& P, int blk) {
    using C = GradKV<HD>;
    constexpr int QT = C::kQueries, NC = C::kCols;
    constexpr uint64_t kTileU = C::kTileBytes >> 4;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    const Args& a = P.a;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int NS = P.kv_stages;           // even: Q and dO tiles in turn
    uint8_t* sK = smem;                   // at the end the rows of dk and dv
    uint8_t* sV = sK + C::kOwnBytes;
    uint8_t* sR = sV + C::kOwnBytes;
    uint8_t* sRow = sR + NS * C::kTileBytes;       // [NS / 2][kRowBytes], the queries' row values
    uint8_t* sOnes = sRow + NS / 2 * kRowBytes;    // [128][8 zeros, 1 1 1 0 0 0 0 0, 8 zeros]
    GradBars& bar = *reinterpret_cast<GradBars*>(sOnes + kOnesBytes);
    float* sBias = reinterpret_cast<float*>(&bar + 1);

    const int split = blk % P.k_splits;
    blk /= P.k_splits;
    const int kt = blk % P.k_tiles;
    blk /= P.k_tiles;
    const int g = blk % a.G;
    const int b = blk / a.G;
    const int j0 = kt * kTile;
    const int end = key_end(a, b);
    uint4 w = make_uint4(0, 0, 0, 0);
    if (j0 < end) w = tile_words(P.kt, b, kt, end);
    const bool any = (w.x | w.y | w.z | w.w) != 0;
    const int64_t pos = a.q_pos ? (int64_t)__ldg(a.q_pos + b) : 0;
    const int dsteps = (a.d + 15) >> 4, dpairs = (a.d + 31) >> 5;
    const int per_head = (a.n + QT - 1) / QT;        // query tiles of a head
    const int nt_all = any ? a.R * per_head : 0, per = (nt_all + P.k_splits - 1) / P.k_splits;
    const int t0 = min(nt_all, split * per), nt = min(nt_all, t0 + per) - t0;

    if (warp == kLoad) {
        if (lane < NS) mbar_init(&bar.full[lane], 1);
        if (lane == NS) mbar_init(&bar.ready, 1);
        fence_mbar_init();
        __syncwarp();
    } else if (warp == kClean) {
        if (lane < NS) {
            mbar_init(&bar.empty[lane], 1);
        } else if (lane == NS) {
            mbar_init(&bar.sfull[0], 1);
            mbar_init(&bar.dpfull[0], 1);
            mbar_init(&bar.pfull, kElemWarps);
            mbar_init(&bar.dsfull[0], kElemWarps);
            mbar_init(&bar.dvdone, 1);
            mbar_init(&bar.done, 1);
            mbar_init(&bar.drain, 1);
        }
        fence_mbar_init();
    }
    if (warp == kIssue) tmem_alloc(&bar.tmem, 512);
    // Q tiles (with the row values of their queries) and dO tiles in turn
    const auto load = [&](int it, int slot) {
        const int t = t0 + (it >> 1), h = g * a.R + t / per_head, qt = t % per_head;
        const bool second = it & 1;
        const TensorMap& src = second ? P.dout : P.q;
        mbar_arrive_expect_tx(&bar.full[slot], C::kTileBytes + (second ? 0 : kRowBytes));
        for (int c = 0; c < C::kChunks; ++c)
            tma_load(sR + slot * C::kTileBytes + c * C::kChunkBytes, &src.map, c * 64, qt * QT, h * src.head,
                     b * src.batch, &bar.full[slot]);
        if (!second)
            bulk_g2s(sRow + (slot >> 1) * kRowBytes,
                     P.rows + (((int64_t)b * a.H + h) * P.q_tiles + qt) * kRowStride, kRowBytes,
                     &bar.full[slot]);
    };
    const int early = min(2 * nt, NS);
    if (warp == kLoad && nt > 0 && elect_one()) {
        mbar_arrive_expect_tx(&bar.ready, 2 * C::kOwnBytes);
        for (int c = 0; c < C::kChunks; ++c) {
            tma_load(sK + c * CHUNK_BYTES, &P.k.map, c * 64, j0, g * P.k.head, b * P.k.batch, &bar.ready);
            tma_load(sV + c * CHUNK_BYTES, &P.v.map, c * 64, j0, g * P.v.head, b * P.v.batch, &bar.ready);
        }
        for (int it = 0; it < early; ++it) load(it, it);
    }
    for (int e = threadIdx.x; e < kOnesBytes / 16; e += kGradThreads)
        reinterpret_cast<uint4*>(sOnes)[e] =
            (e / 8) % 3 == 1 ? make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;

    if (warp == kLoad) {
        if (nt > 0 && elect_one()) {
            Ring r;
            r.step(early, NS);
            int issued = early;
            bool ok = true;
            for (int it = early; it < 2 * nt; ++it) {
                if (!mbar_wait(&bar.empty[r.slot], r.phase ^ 1u, a.err, ERR_TIMEOUT_PRODUCER)) {
                    ok = false;
                    break;
                }
                load(it, r.slot);
                ++issued;
                r.step(1, NS);
            }
            if (!ok) {
                mbar_wait(&bar.ready, 0, a.err, ERR_TIMEOUT_PRODUCER);
                Ring l;
                for (int it = 0; it < issued; ++it) {
                    if (it + NS >= issued)
                        mbar_wait(&bar.full[l.slot], l.phase, a.err, ERR_TIMEOUT_PRODUCER);
                    l.step(1, NS);
                }
            }
        }
    } else if (warp == kIssue) {
        if (nt > 0 && elect_one()) {
            const uint32_t idS = idesc_16(BF, kTile, false);
            const uint32_t idD = idesc_16(BF, dsteps * 16, true);
            const uint64_t dK = sdesc_sw128(smem_u32(sK)), dV = sdesc_sw128(smem_u32(sV));
            const uint64_t dR = sdesc_sw128(smem_u32(sR)), dRt = sdesc_tokens(smem_u32(sR));
            const uint32_t idR = idesc_16(true, kTile, false);
            const uint64_t dRow = sdesc_flat(smem_u32(sRow), 128, 256);
            const uint64_t dOnes = sdesc_flat(smem_u32(sOnes), 128, 384);
            Ring rs, rd;      // tiles whose scores, and whose dV and dK, come next: Q at slot, dO at slot + 1
            // K Q^T - lse2 / scale2, V dO^T - delta: the row values are a last product's sums
            const auto scores = [&]() {
                mma_over_d<2>(tmem + C::S, dK, dR + rs.slot * kTileU, idS, dpairs);
                mma_f16(tmem + C::S, dOnes + (128 >> 4), dRow + (rs.slot >> 1) * (kRowBytes >> 4), idR, true);
                mma_commit(&bar.sfull[0]);
            };
            const auto grads = [&]() {
                mma_over_d<2>(tmem + C::DP, dV, dR + (rs.slot + 1) * kTileU, idS, dpairs);
                mma_f16(tmem + C::DP, dOnes, dRow + (rs.slot >> 1) * (kRowBytes >> 4), idR, true);
                mma_commit(&bar.dpfull[0]);
                rs.step(2, NS);
            };
            bool ok = mma_wait(a.err, &bar.ready, 0) && mma_wait(a.err, &bar.full[0], 0);
            if (ok) {
                scores();
                ok = mma_wait(a.err, &bar.full[1], 0);
            }
            if (ok) grads();
            for (int t = 0; t < nt && ok; ++t) {
                const bool more = t + 1 < nt;
                const bool p_seen = mbar_test(&bar.pfull, t & 1);
                const bool q_seen = more && mbar_test(&bar.full[rs.slot], rs.phase);
                const bool do_seen = more && mbar_test(&bar.full[rs.slot + 1], rs.phase);
                if (!(ok = p_seen || mma_wait(a.err, &bar.pfull, t & 1))) break;
                tc_fence_after();
                mma_over_tokens(tmem + C::DV, tmem + C::S, dRt + (rd.slot + 1) * kTileU, idD, t > 0, 64);
                mma_commit(more ? &bar.empty[rd.slot + 1] : &bar.dvdone);
                if (more) {
                    if (!(ok = q_seen || mma_wait(a.err, &bar.full[rs.slot], rs.phase))) break;
                    scores();
                }
                if (!(ok = mma_wait(a.err, &bar.dsfull[0], t & 1))) break;
                mma_over_tokens(tmem + C::DK, tmem + C::DP, dRt + rd.slot * kTileU, idD, t > 0, 64);
                mma_commit(&bar.empty[rd.slot]);
                rd.step(2, NS);
                if (more) {
                    if (!(ok = do_seen || mma_wait(a.err, &bar.full[rs.slot + 1], rs.phase))) break;
                    grads();
                }
            }
            mma_commit(&bar.done);
            mma_commit(&bar.drain);
            mbar_wait(&bar.drain, 0, a.err, ERR_TIMEOUT_MMA);
        }
    } else if (warp < kElemWarps) {
        const int quarter = warp & 3, half = warp >> 2;
        const int r = quarter * 32 + lane;
        const int j = j0 + r;
        const uint32_t lofs = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + lofs + C::S + half * NC, tDP = tmem + lofs + C::DP + half * NC;
        const float scale2 = least_scale(a);
        // float16: p and ds are 2^kGradShift and 2^shift times as large
        const int shift = BF ? 0 : range_shift(P, b, g * a.R, 0, a.R * P.q_tiles);
        const float ds_over_p = power2(shift - (BF ? 0 : kGradShift));
        bool ok = true;
        int h = g * a.R + t0 / per_head, qt = t0 % per_head;
        for (int t = 0; t < nt; ++t) {
            if (a.table && (qt == 0 || t == 0)) {
                named_sync(1, 32 * kElemWarps);
                fill_bias<BF>(a, h, sBias, threadIdx.x, 32 * kElemWarps);
                named_sync(1, 32 * kElemWarps);
            }
            // (a warp that gave up still meets the others at the barriers above)
            float v[NC];
            ok = ok && warp_wait(&bar.sfull[0], t & 1, a.err, ERR_TIMEOUT_EPILOGUE);
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < NC; c += 32) tmem_ld32(tS + c, v + c);
                tmem_wait_ld();
                tmem_reg_fence(v);
                float mul = scale2, add = 0.f;
                if (a.table) {
                    // relative position of the tile's first key and the strip's first query
                    const int64_t rel0 = (int64_t)j0 - pos - (int64_t)qt * QT - half * NC;
                    if (rel0 - (NC - 1) >= a.D) {
                        add = sBias[2 * a.D + kSlack];
                    } else if (rel0 + (kTile - 1) <= -a.D) {
                        add = sBias[kSlack];
                    } else {
                        const float* e = sBias + (int)rel0 + r + a.D + kSlack;
#pragma unroll
                        for (int c = 0; c < NC; ++c) v[c] = fmaf(v[c], mul, e[-c]);
                        mul = 1.f;
                    }
                }
                if (!BF) add += (float)kGradShift;
                const uint64_t mul2 = pk(mul, mul), add2 = pk(add, add);
#pragma unroll
                for (int c = 0; c < NC; c += 2) {
                    upk(fma2(pk(v[c], v[c + 1]), mul2, add2), v[c], v[c + 1]);
                    v[c] = ex2(v[c]);
                    v[c + 1] = ex2(v[c + 1]);
                }
                {
                    uint32_t u[NC / 2];
#pragma unroll
                    for (int c = 0; c < NC / 2; ++c) u[c] = pack16<BF>(v[2 * c], v[2 * c + 1]);
                    tmem_st32(tS, u);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.pfull);
                }
            }
            ok = ok && warp_wait(&bar.dpfull[0], t & 1, a.err, ERR_TIMEOUT_EPILOGUE);
            if (ok) {
                tc_fence_after();
                uint32_t u[NC / 2];
#pragma unroll
                for (int q = 0; q < NC; q += 32) {
                    float d[32];
                    tmem_ld32(tDP + q, d);
                    tmem_wait_ld();
                    tmem_reg_fence(d);
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        float f0, f1;
                        uint64_t ds = mul2f(pk(v[q + c], v[q + c + 1]), pk(d[c], d[c + 1]));
                        if (!BF) ds = mul2f(ds, pk(ds_over_p, ds_over_p));
                        upk(ds, f0, f1);
                        u[(q + c) / 2] = pack16<BF>(f0, f1);
                    }
                }
                tmem_st32(tDP, u);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.dsfull[0]);
            }
            if (++qt == per_head) {
                qt = 0;
                ++h;
            }
        }
        const uint32_t word = quarter == 0 ? w.x : quarter == 1 ? w.y : quarter == 2 ? w.z : w.w;
        const bool keep = (word >> lane) & 1u;
        const int w0 = j - lane + half * 16, r0 = quarter * 32 + half * 16;
        if (nt > 0 && ok) ok = warp_wait(&bar.dvdone, 0, a.err, ERR_TIMEOUT_EPILOGUE);
        tc_fence_after();
        const bool whole = P.k_splits == 1;
        const int64_t part = ((((int64_t)split * a.B + b) * a.G + g) * a.m + j) * a.d;
        const float dv_scale = BF ? 1.f : power2(-kGradShift);
        const float dk_scale = BF ? a.scale : a.scale * power2(-shift);
        if (ok && whole)
            stage_row<HD, BF>(sV, r, tmem + lofs + C::DV, half, dsteps, dv_scale, nt > 0, keep);
        else if (ok)
            part_row<HD>(P.part_dv + part, j < a.m, tmem + lofs + C::DV, half, dsteps, dv_scale, nt > 0, a.d);
        named_sync(2 + quarter, 64);
        if (ok && whole)
            unstage_rows<16>(sV, r0, a.m - w0, a.d,
                             static_cast<uint16_t*>(a.dv.p) + b * a.dv.sb + (int64_t)w0 * a.dv.st + g * a.dv.sh,
                             a.dv.st, P.dv_vec, lane);
        if (nt > 0 && ok) ok = warp_wait(&bar.done, 0, a.err, ERR_TIMEOUT_EPILOGUE);
        tc_fence_after();
        if (ok && whole)
            stage_row<HD, BF>(sK, r, tmem + lofs + C::DK, half, dsteps, dk_scale, nt > 0, keep);
        else if (ok)
            part_row<HD>(P.part_dk + part, j < a.m, tmem + lofs + C::DK, half, dsteps, dk_scale, nt > 0, a.d);
        named_sync(2 + quarter, 64);
        if (ok && whole)
            unstage_rows<16>(sK, r0, a.m - w0, a.d,
                             static_cast<uint16_t*>(a.dk.p) + b * a.dk.sb + (int64_t)w0 * a.dk.st + g * a.dk.sh,
                             a.dk.st, P.dk_vec, lane);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kIssue) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Both in one launch: the blocks of the keys, which take longer, first; those of the
// queries fill the GPU's last wave.
template <int HD, bool BF>
__global__ void __launch_bounds__(kGradThreads, 1) k_grad(const __grid_constant__ GradArgs P) {
    const int keys = P.k_tiles * P.a.G * P.a.B * P.k_splits;
    if ((int)blockIdx.x < keys)
        grad_keys<HD, BF>(P, blockIdx.x);
    else
        grad_queries<HD, BF, false>(P, blockIdx.x - keys);
}

template <int HD, bool BF>
__global__ void __launch_bounds__(kGradThreads, 1) k_grad_delta(const __grid_constant__ GradArgs P) {
    grad_queries<HD, BF, true>(P, blockIdx.x);
}

// The shares of a gradient added in their order: a row (b, head, token) a warp.  A key that
// does not count has a zero gradient whatever its row holds.
template <bool BF>
__global__ void __launch_bounds__(128) k_grad_join(Args a, View w, View w1, const float* part, const float* part1,
                                                   int splits, int tokens, int heads,
                                                   const uint4* __restrict__ words, int tiles, bool keys) {
    if (blockIdx.y) {
        w = w1;
        part = part1;
    }
    const int64_t rows = (int64_t)a.B * heads * tokens, row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const int t = (int)(row % tokens), h = (int)(row / tokens % heads), b = (int)(row / tokens / heads);
    bool counts = true;
    if (keys) {
        counts = t < key_end(a, b);
        if (counts && words) {
            const uint32_t* u = reinterpret_cast<const uint32_t*>(words + (int64_t)b * tiles + t / kTile);
            counts = (u[(t % kTile) / 32] >> (t % 32)) & 1u;
        }
    }
    Elem<BF>* out = static_cast<Elem<BF>*>(w.p) + b * w.sb + (int64_t)t * w.st + h * w.sh;
    for (int c = lane; c < a.d; c += 32) {
        float s = 0.f;
        if (counts)
#pragma unroll 8
            for (int k = 0; k < splits; ++k) s += __ldg(part + (k * rows + row) * a.d + c);
        out[c] = from_f<Elem<BF>>(s);
    }
}

// Row values of the queries from the shares of delta: a row a thread.
template <bool BF>
__global__ void __launch_bounds__(kTile) k_delta_join(const __grid_constant__ GradArgs P) {
    const Args& a = P.a;
    int blk = blockIdx.x;
    const int qt = blk % P.q_tiles;
    blk /= P.q_tiles;
    const int h = blk % a.H, b = blk / a.H, r = threadIdx.x;
    const int64_t tile = (int64_t)blockIdx.x;
    float s = 0.f, top = 0.f;
    for (int k = 0; k < P.q_splits; ++k) {
        const int64_t at = (k * (int64_t)gridDim.x + tile) * kTile + r;
        s += P.part_delta[at];
        if (!BF) top = fmaxf(top, P.part_top[at]);
    }
    uint8_t* values = P.rows + tile * kRowStride;
    put_row(a, values, r, -s, true);
    put_row(a, values, r, row_lse(a, b, h, (int64_t)qt * kTile + r), false);
    if (!BF) put_range(P, tile, r >> 5, r & 31, top + fabsf(s));
}

// ---------------------------------------------------------------------------
// dbias of one row of the table: the blocks' sums by relative position, in
// their order, then the positions of each bucket in theirs.

constexpr int kBiasThreads = 1024;
constexpr int kBiasSplit = 8;      // most shares of the blocks' sums

template <bool BF>
__global__ void __launch_bounds__(kBiasThreads) k_grad_bias(const __grid_constant__ GradArgs P, int shares,
                                                            Elem<BF>* __restrict__ dbias) {
    extern __shared__ float sSum[];                 // [shares][width], then the buckets
    const Args& a = P.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int width = 2 * a.D + 1;
    int* sBucket = reinterpret_cast<int*>(sSum + shares * width);
    const int64_t parts = (int64_t)a.B * P.q_tiles * P.q_splits * (a.table_stride ? 1 : a.H);
    const float* src = a.bias_part + blockIdx.x * parts * width;
    const int64_t per = (parts + shares - 1) / shares;
    const int strips = (width + 31) / 32;
    for (int x = warp; x < strips * shares; x += kBiasThreads / 32) {
        const int share = x / strips, e = (x % strips) * 32 + lane;
        if (e >= width) continue;
        const int64_t p0 = share * per, p1 = min(parts, p0 + per);
        float s = 0.f;
#pragma unroll 16
        for (int64_t p = p0; p < p1; ++p) s += src[p * width + e];
        sSum[share * width + e] = s;
    }
    for (int e = threadIdx.x; e < width; e += kBiasThreads) sBucket[e] = bucket_of(a, e - a.D);
    __syncthreads();
    for (int e = threadIdx.x; e < width; e += kBiasThreads) {
        float s = sSum[e];
        for (int k = 1; k < shares; ++k) s += sSum[k * width + e];
        sSum[e] = s;
    }
    __syncthreads();
    for (int u = warp; u < a.nb; u += kBiasThreads / 32) {
        float s = 0.f;
        for (int e = lane; e < width; e += 32)
            if (sBucket[e] == u) s += sSum[e];
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) dbias[(int64_t)blockIdx.x * a.nb + u] = from_f<Elem<BF>>(s);
    }
}

// ---------------------------------------------------------------------------

int ring_stages(size_t fixed, size_t per_stage) {
    const int s = (int)((kSmemLimit - fixed) / per_stage);
    return s < kMaxRing ? s : kMaxRing;
}

// the least shared memory of the largest calls leaves four tiles
static_assert(1024 + sizeof(GradBars) + 4 * 2 * kElemWarps + 4 * (2 * (kMaxDistance + kSlack) + 1) +
                      4 * kBands * (2 * kMaxDistance + 1) + 4 * kElemWarps * 8 * 33 + 4 * 2 * CHUNK_BYTES <=
                  kSmemLimit,
              "grad_queries does not fit in shared memory");
static_assert(1024 + sizeof(GradBars) + 4 * (2 * (kMaxDistance + kSlack) + 1) + kOnesBytes +
                      6 * 2 * CHUNK_BYTES + 2 * kRowBytes <=
                  kSmemLimit,
              "grad_keys does not fit in shared memory");

template <int HD, bool BF>
cudaError_t launch_grad(GradArgs p, void* dbias, cudaStream_t s) {
    const Args& a = p.a;
    using Q = GradQ<HD>;
    using KV = GradKV<HD>;
    const size_t bias = a.table ? sizeof(float) * (2 * (size_t)(a.D + kSlack) + 1) : 0;
    const size_t width = 2 * (size_t)a.D + 1;
    static std::atomic<uint64_t> ready{0}, delta_ready{0};
    cudaError_t e;
    size_t fixed = 1024 + sizeof(GradBars) + sizeof(float) * 2 * kElemWarps + bias +
                   (a.bias_part ? sizeof(float) * kBands * width : 0);
    // shared memory for the diagonals of ds, 32 rows at a time.  16 where that leaves six
    // tiles in flight instead of four, so that the next key tile has landed in time (batch
    // 4, 2048 x 2048, 16 heads of 128, distance 128: 453 us for 501); 8 where fewer than
    // the four are left that the order of the products needs (distances from about 1500)
    const auto scratch = [&](int rows) { return a.bias_part ? sizeof(float) * kElemWarps * rows * 33 : 0; };
    const auto stages = [&](int rows) { return ring_stages(fixed + scratch(rows), Q::kTileBytes); };
    p.scratch_rows = stages(32) >= 6 ? 32 : stages(16) >= 6 ? 16 : stages(32) >= 4 ? 32 : 8;
    fixed += scratch(p.scratch_rows);
    p.stages = 2 * (ring_stages(fixed, Q::kTileBytes) / 2);
    size_t smem = fixed + p.stages * Q::kTileBytes;
    // K and V, then stages of which each pair has the row values of its queries
    constexpr size_t stage = KV::kTileBytes + kRowBytes / 2;
    fixed = 1024 + sizeof(GradBars) + bias + 2 * KV::kOwnBytes + kOnesBytes;
    p.kv_stages = 2 * (ring_stages(fixed, stage) / 2);
    smem = std::max(smem, fixed + p.kv_stages * stage);
    if ((e = raise_smem(k_grad<HD, BF>, kSmemLimit, ready)) != cudaSuccess) return e;
    const int64_t q_blocks = (int64_t)p.q_tiles * a.H * a.B, k_blocks = (int64_t)p.k_tiles * a.G * a.B;
    if (p.exact_delta) {
        const size_t least = 1024 + sizeof(GradBars) + sizeof(float) * 2 * kTile + bias;
        p.delta_stages = 2 * (ring_stages(least, Q::kTileBytes) / 2);
        if ((e = raise_smem(k_grad_delta<HD, BF>, kSmemLimit, delta_ready)) != cudaSuccess) return e;
        k_grad_delta<HD, BF><<<(unsigned)(q_blocks * p.q_splits), kGradThreads,
                               least + p.delta_stages * Q::kTileBytes, s>>>(p);
        if (p.q_splits > 1) {
            k_delta_join<BF><<<(unsigned)q_blocks, kTile, 0, s>>>(p);
            count_launch();
        }
    } else {
        k_grad_rows<HD / 8, BF><<<(unsigned)(q_blocks + (BF ? 0 : k_blocks)), kRowThreads, 0, s>>>(p);
    }
    count_launch();
    k_grad<HD, BF><<<(unsigned)(q_blocks * p.q_splits + k_blocks * p.k_splits), kGradThreads, smem, s>>>(p);
    count_launch();
    const auto join = [&](const View& w, const View& w1, const float* part, const float* part1, int splits,
                          int tokens, int heads, bool keys) {
        const dim3 grid((unsigned)(((int64_t)a.B * heads * tokens + 3) / 4), keys ? 2 : 1);
        k_grad_join<BF><<<grid, 128, 0, s>>>(a, w, w1, part, part1, splits, tokens, heads, p.kt.words, p.kt.tiles,
                                             keys);
        count_launch();
    };
    if (p.q_splits > 1) join(a.dq, a.dq, p.part_dq, p.part_dq, p.q_splits, a.n, a.H, false);
    if (p.k_splits > 1) join(a.dk, a.dv, p.part_dk, p.part_dv, p.k_splits, a.m, a.G, true);
    if (dbias) {
        // shares of the sums and the buckets in 48 KB; no more than the warps take in one turn
        const int strips = (int)(width + 31) / 32;
        const int shares =
            std::max(1, std::min({kBiasSplit, (int)(12288 / width) - 1, kBiasThreads / 32 / strips}));
        k_grad_bias<BF><<<a.table_stride ? a.H : 1, kBiasThreads, 4 * (shares + 1) * width, s>>>(
            p, shares, static_cast<Elem<BF>*>(dbias));
        count_launch();
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grad_tc(const GradArgs& p, void* dbias, cudaStream_t s) {
    if (p.a.d <= 64) return p.a.bf16 ? launch_grad<64, true>(p, dbias, s) : launch_grad<64, false>(p, dbias, s);
    return p.a.bf16 ? launch_grad<128, true>(p, dbias, s) : launch_grad<128, false>(p, dbias, s);
}

}  // namespace attn
}  // namespace fs
