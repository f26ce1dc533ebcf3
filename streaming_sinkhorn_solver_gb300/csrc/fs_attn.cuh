// Shared declarations of the cross-attention kernels.
//
// Notation: z_ij = scale q_i . k_j + bias in base 2 is x_ij = z_ij log2(e), so
// p_ij = 2^{x_ij - lse2_i} with lse2_i = lse_i log2(e).  Tokens are numbered
// within their sequence; query head h reads key head h / R, R = heads / kv_heads.
#pragma once

#include "fs_internal.cuh"

#include <cuda_bf16.h>

namespace fs {
namespace attn {

constexpr int kMaxHeadDim = 128;
constexpr int kMaxBuckets = 1024;
constexpr int kMaxDistance = 2048;

// a (batch, token, head, d) tensor: element strides, the d elements contiguous
struct View {
    void* p;
    int64_t sb, st, sh;
};

struct Args {
    View q, k, v, o, dout, dq, dk, dv;
    int B, H, G, R, n, m, d;
    int bf16;                    // 1 bfloat16, 0 float16
    float scale, scale2;         // scale, scale log2(e)
    float* lse;                  // [B][H][n], natural logarithm
    const int32_t* kv_len;       // [B] or nullptr
    const uint8_t* mask;         // rows of m or nullptr
    int64_t mask_stride;
    const void* table;           // bias rows or nullptr
    int64_t table_stride;
    const int32_t* buckets;      // [2 D + 1]
    int nb, D;
    const int32_t* q_pos;        // [B] or nullptr
    float* bias_part;            // [H][B][query tiles][2 D + 1] sums of the bias gradient, or nullptr
    uint32_t* err;               // device error word
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// counted keys end: kv_len[b] taken into [0, m]
__device__ __forceinline__ int key_end(const Args& a, int b) {
    if (a.kv_len == nullptr) return a.m;
    const int l = __ldg(a.kv_len + b);
    return l < 0 ? 0 : (l < a.m ? l : a.m);
}

__device__ __forceinline__ int bucket_of(const Args& a, int64_t rel) {
    const int64_t r = rel < -a.D ? -a.D : (rel > a.D ? a.D : rel);
    const int u = __ldg(a.buckets + (r + a.D));
    return u < 0 ? 0 : (u < a.nb ? u : a.nb - 1);
}

// bias entry in base 2; entries below -1e30 (bfloat16's lowest value stands for
// "never" in additive masks) forbid their pairs as -inf does, so that such
// rows stay empty instead of losing their scores to rounding.  float16 ends at -65504, a
// number like others: a row that has no other bias keeps its scores to 2^-7 in base 2.
__device__ __forceinline__ float bias2(float v) {
    return v < -1e30f ? -INFINITY : v * (float)kLog2e;
}

}  // namespace attn
}  // namespace fs
