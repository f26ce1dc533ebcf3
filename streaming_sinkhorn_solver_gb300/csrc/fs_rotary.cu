// Rotary positions of queries and keys, and their gradient (the same turned back).
//
// Bound by memory: every element is read and written once.  A block takes up to 8 tokens:
// first the frequencies, then the sines and cosines of each token into shared memory, where
// all their heads find them, then the heads, 16 bytes an access.  Measured: 2 x 8192 tokens of
// 40 heads of 128, bfloat16: 58 us, 5.7 TB/s (0.85 of the measured copy rate); 3 x 2777 tokens of
// 28 heads of 80, pairs of neighbours, half of the head, with the gradient: 35 us, 4.3 TB/s.
//
// Angles.  A frequency is kept as a 64-bit fraction of a turn, F = frac(w / 2 pi) 2^64, so
// that a position's angle is the low 64 bits of p F: whole turns fall away by themselves,
// with no reduction and no double arithmetic per token (a type that this GPU has next to no
// units for).  w / 2 pi is formed in two doubles, as one would be off by 2^-53 of it, which at
// position 2^31 is 2^-22 turns for each turn a position and many for a w of 10^6.  So is F by
// half of 2^-64 for |w| below 2^40, and a position's angle by 2^-32 turns, cut from p F.
#include "fs_attn_host.cuh"

#include <algorithm>
#include <cmath>

namespace fs {
namespace rotary {

namespace {

using attn::View;

constexpr int kThreads = 128;
constexpr int kTokens = 8;             // most tokens of a block
constexpr int kMaxRotary = 512;

struct Args {
    View x[2], y[2];             // queries and keys: input, output
    int heads[2];
    int B, n, d, half;
    float amplitude;
    const double* freqs;
    const int32_t* pos;
    int64_t pos_b, pos_t;
    int tokens;                  // of a block
    int back;                    // turned back
    int vec;                     // every row takes 16-byte accesses
};

template <typename T>
__device__ __forceinline__ void unpack(uint32_t w, float& x, float& y) {
    const uint16_t a = (uint16_t)w, b = (uint16_t)(w >> 16);
    x = attn::to_f<T>(*reinterpret_cast<const T*>(&a));
    y = attn::to_f<T>(*reinterpret_cast<const T*>(&b));
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float x, float y) {
    const T a = attn::from_f<T>(x), b = attn::from_f<T>(y);
    return (uint32_t)*reinterpret_cast<const uint16_t*>(&b) << 16 | *reinterpret_cast<const uint16_t*>(&a);
}

// x less whole numbers, in 2^-64
__device__ __forceinline__ uint64_t fraction(double x) { return (uint64_t)__double2ll_rn((x - rint(x)) * 0x1p64); }

// PAIRS: neighbours (2 i, 2 i + 1) are pairs, else (i, i + half)
template <typename T, bool PAIRS>
__global__ void __launch_bounds__(kThreads) k_rotary(const __grid_constant__ Args P) {
    extern __shared__ __align__(16) float2 turn[];     // [tokens][half] amplitude (cos, sin)
    __shared__ uint64_t step[kMaxRotary / 2];
    __shared__ float amplitude[kMaxRotary / 2];        // NaN for a frequency that is not finite
    __shared__ int32_t place[kTokens];
    __shared__ int64_t at[kTokens][4];       // where a token's queries and keys begin: input, output
    const int64_t all = (int64_t)P.B * P.n;
    const int64_t first = (int64_t)blockIdx.x * P.tokens;
    const int count = (int)min((int64_t)P.tokens, all - first);
    for (int i = threadIdx.x; i < P.half; i += kThreads) {
        constexpr double kHigh = 0x1.45f306dc9c883p-3, kLow = -0x1.6b01ec5417056p-57;      // 1 / 2 pi
        const double w = __ldg(P.freqs + i), turns = w * kHigh;
        step[i] = fraction(turns) + fraction(fma(w, kLow, fma(w, kHigh, -turns)));
        amplitude[i] = isfinite(w) ? P.amplitude : __int_as_float(0x7fc00000);
    }
    if (threadIdx.x < count) {
        const unsigned tok = (unsigned)(first + threadIdx.x), b = tok / (unsigned)P.n;
        const int64_t i = tok - b * (unsigned)P.n;
        place[threadIdx.x] = __ldg(P.pos + b * P.pos_b + i * P.pos_t);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            at[threadIdx.x][k] = b * P.x[k].sb + i * P.x[k].st;
            at[threadIdx.x][2 + k] = b * P.y[k].sb + i * P.y[k].st;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < count * P.half; e += kThreads) {
        const int t = e / P.half, i = e - t * P.half;
        const int64_t p = place[t];
        const int32_t top = (int32_t)(((uint64_t)p * step[i]) >> 32);
        float sn, cs;
        sincospif((float)top * 0x1p-31f, &sn, &cs);
        turn[e] = make_float2(amplitude[i] * cs, amplitude[i] * (P.back ? -sn : sn));
    }
    __syncthreads();
    const int heads = P.heads[0] + P.heads[1];
    if (P.vec) {
        // Units of a head: the turned ones (8 elements, or 8 of each half), then copies of 8.  A
        // thread takes one of a head for kUnits tokens at a time, whose loads are under way together.
        constexpr int kUnits = 4;
        const int turned = PAIRS ? P.half / 4 : P.half / 8;
        const int units = turned + (P.d - 2 * P.half) / 8;
        for (int e = threadIdx.x; e < heads * units; e += kThreads) {
            int h = e / units;
            const int u = e - h * units;
            const int which = h >= P.heads[0];
            if (which) h -= P.heads[0];
            const bool turns = u < turned;
            const int c = turns ? 8 * u : 2 * P.half + 8 * (u - turned);
            const uint16_t* src = static_cast<const uint16_t*>(P.x[which].p) + h * P.x[which].sh + c;
            uint16_t* dst = static_cast<uint16_t*>(P.y[which].p) + h * P.y[which].sh + c;
            const float2* w = turn + (PAIRS ? 4 * u : 8 * u);
            for (int t0 = 0; t0 < count; t0 += kUnits) {
                uint4 x[kUnits], y[kUnits];
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    if (t0 + i >= count) break;
                    const uint16_t* p = src + at[t0 + i][which];
                    x[i] = *reinterpret_cast<const uint4*>(p);
                    if (!PAIRS && turns) y[i] = *reinterpret_cast<const uint4*>(p + P.half);
                }
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    if (t0 + i >= count) break;
                    uint16_t* to = dst + at[t0 + i][2 + which];
                    const float2* z0 = w + (t0 + i) * P.half;
                    uint32_t o[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    if (turns && PAIRS) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float a, c1;
                            unpack<T>(o[k], a, c1);
                            const float2 z = z0[k];
                            o[k] = pack<T>(a * z.x - c1 * z.y, a * z.y + c1 * z.x);
                        }
                    } else if (turns) {
                        uint32_t r[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float a0, a1, c0, c1;
                            unpack<T>(o[k], a0, a1);
                            unpack<T>(r[k], c0, c1);
                            const float4 z = reinterpret_cast<const float4*>(z0)[k];
                            o[k] = pack<T>(a0 * z.x - c0 * z.y, a1 * z.z - c1 * z.w);
                            r[k] = pack<T>(a0 * z.y + c0 * z.x, a1 * z.w + c1 * z.z);
                        }
                        *reinterpret_cast<uint4*>(to + P.half) = make_uint4(r[0], r[1], r[2], r[3]);
                    }
                    *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
        return;
    }
    // one pair, or one element behind the pairs, a thread
    const int units = P.d - P.half;
    for (int e = threadIdx.x; e < count * heads * units; e += kThreads) {
        const int row = e / units, u = e - row * units;
        const int t = row / heads;
        int h = row - t * heads;
        const int which = h >= P.heads[0];
        if (which) h -= P.heads[0];
        const T* src = static_cast<const T*>(P.x[which].p) + at[t][which] + h * P.x[which].sh;
        T* dst = static_cast<T*>(P.y[which].p) + at[t][2 + which] + h * P.y[which].sh;
        if (u >= P.half) {
            dst[P.half + u] = src[P.half + u];
            continue;
        }
        const int c0 = PAIRS ? 2 * u : u, c1 = PAIRS ? 2 * u + 1 : u + P.half;
        const float a = attn::to_f<T>(src[c0]), c = attn::to_f<T>(src[c1]);
        const float2 z = turn[t * P.half + u];
        dst[c0] = attn::from_f<T>(a * z.x - c * z.y);
        dst[c1] = attn::from_f<T>(a * z.y + c * z.x);
    }
}

template <typename T>
cudaError_t launch(const Args& p, bool pairs, cudaStream_t s) {
    const int64_t blocks = ((int64_t)p.B * p.n + p.tokens - 1) / p.tokens;
    const size_t smem = sizeof(float2) * (size_t)p.tokens * p.half;
    if (pairs)
        k_rotary<T, true><<<(unsigned)blocks, kThreads, smem, s>>>(p);
    else
        k_rotary<T, false><<<(unsigned)blocks, kThreads, smem, s>>>(p);
    count_launch();
    return cudaGetLastError();
}

fs_status rotary_entry(const fs_rotation* r, const void* q, const void* k, void* q_out, void* k_out,
                       void* stream, bool back) {
    if (!r) return fail(FS_ERR_INVALID_ARG, "null fs_rotation");
    if (r->dtype != FS_DTYPE_BF16 && r->dtype != FS_DTYPE_F16)
        return fail(FS_ERR_INVALID_ARG, "fs_rotation.dtype=%d", r->dtype);
    constexpr int kMostHeads = 1 << 16;
    if (r->heads < 1 || r->heads > kMostHeads || r->kv_heads < 0 || r->kv_heads > kMostHeads)
        return fail(FS_ERR_INVALID_ARG, "heads=%d kv_heads=%d out of range", r->heads, r->kv_heads);
    if (r->d < 1 || r->d > 4096) return fail(FS_ERR_INVALID_ARG, "d=%d out of range [1, 4096]", r->d);
    if (r->rotary_dim < 2 || r->rotary_dim % 2 || r->rotary_dim > r->d || r->rotary_dim > kMaxRotary)
        return fail(FS_ERR_INVALID_ARG, "rotary_dim=%d is not even in [2, min(d, %d)]", r->rotary_dim,
                    kMaxRotary);
    if (r->interleaved != 0 && r->interleaved != 1)
        return fail(FS_ERR_INVALID_ARG, "interleaved=%d", r->interleaved);
    constexpr int64_t kMaxTokens = INT32_MAX - 4096;
    if (r->batch < 0 || r->n < 0 || r->batch > kMaxTokens || r->n > kMaxTokens)
        return fail(FS_ERR_INVALID_ARG, "batch=%lld n=%lld out of range [0, %lld]", (long long)r->batch,
                    (long long)r->n, (long long)kMaxTokens);
    if (!std::isfinite(r->amplitude)) return fail(FS_ERR_INVALID_ARG, "amplitude must be finite");
    if (r->reserved) return fail(FS_ERR_INVALID_ARG, "fs_rotation.reserved must be zero");
    if (r->pos_stride[0] < 0 || r->pos_stride[1] < 0)
        return fail(FS_ERR_INVALID_ARG, "pos has a negative stride");
    const int dev = attn::current_device();
    Args p = {};
    FS_TRY(attn::view(dev, p.x[0], q, r->q_stride, r->batch, r->n, r->heads, r->d, false, "q"));
    FS_TRY(attn::view(dev, p.y[0], q_out, r->q_out_stride, r->batch, r->n, r->heads, r->d, true, "q_out"));
    if (r->kv_heads) {
        FS_TRY(attn::view(dev, p.x[1], k, r->k_stride, r->batch, r->n, r->kv_heads, r->d, false, "k"));
        FS_TRY(attn::view(dev, p.y[1], k_out, r->k_out_stride, r->batch, r->n, r->kv_heads, r->d, true,
                          "k_out"));
    }
    const int64_t tokens = r->batch * r->n;
    FS_TRY(attn::check_ptr(dev, r->freqs, 1, "freqs"));
    FS_TRY(attn::check_ptr(dev, r->pos, tokens, "pos"));
    if ((double)r->batch * r->n > (double)kMaxTokens)
        return fail(FS_ERR_UNSUPPORTED, "%.3g tokens in one call", (double)r->batch * r->n);
    if (tokens == 0) return FS_OK;
    p.heads[0] = r->heads;
    p.heads[1] = r->kv_heads;
    p.B = (int)r->batch;
    p.n = (int)r->n;
    p.d = r->d;
    p.half = r->rotary_dim / 2;
    p.amplitude = r->amplitude;
    p.freqs = r->freqs;
    p.pos = r->pos;
    p.pos_b = r->pos_stride[0];
    p.pos_t = r->pos_stride[1];
    p.back = back;
    // the turned part and each half of it in whole pieces of 16 bytes
    p.vec = p.d % 8 == 0 && (r->interleaved ? p.half % 4 == 0 : p.half % 8 == 0);
    for (int w = 0; w < (r->kv_heads ? 2 : 1); ++w)
        p.vec = p.vec && attn::aligned16(p.x[w], p.B, p.n, p.heads[w]) &&
                attn::aligned16(p.y[w], p.B, p.n, p.heads[w]);
    // the frequencies of a block's tokens are brought into shape once: as many as leave the GPU full
    p.tokens = (int)std::min<int64_t>(kTokens, std::max<int64_t>(1, tokens / 1024));
    NvtxRange range(back ? "fs_rotary_grad" : "fs_rotary");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    FS_CUDA(r->dtype == FS_DTYPE_BF16 ? launch<__nv_bfloat16>(p, r->interleaved, s)
                                      : launch<__half>(p, r->interleaved, s));
    return FS_OK;
}

}  // namespace

}  // namespace rotary
}  // namespace fs

using namespace fs;

extern "C" {

fs_status fs_rotary(const fs_rotation* rot, const void* q, const void* k, void* q_out,
                    void* k_out, void* stream) {
    try {
        return rotary::rotary_entry(rot, q, k, q_out, k_out, stream, false);
    } catch (...) {
        return fail(FS_ERR_CUDA, "unexpected host exception");
    }
}

fs_status fs_rotary_grad(const fs_rotation* rot, const void* dq, const void* dk, void* dq_out,
                         void* dk_out, void* stream) {
    try {
        return rotary::rotary_entry(rot, dq, dk, dq_out, dk_out, stream, true);
    } catch (...) {
        return fail(FS_ERR_CUDA, "unexpected host exception");
    }
}

}  // extern "C"
