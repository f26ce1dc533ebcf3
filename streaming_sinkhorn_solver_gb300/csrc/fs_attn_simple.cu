// Cross attention, the plain form on the GPU: one block per query row (or key
// row, for dk and dv), one key (query) per thread and step, then one of the d
// coordinates per thread.  Every sum is float32 and every order fixed.
#include "fs_attn.cuh"

namespace fs {
namespace attn {

namespace {

constexpr int kT = 128;   // threads, keys per step, and the most coordinates of a head

__device__ __forceinline__ float block_max(float x, float* sh) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    return fmaxf(fmaxf(sh[0], sh[1]), fmaxf(sh[2], sh[3]));
}

__device__ __forceinline__ float block_sum(float x, float* sh) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    return (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

template <typename T>
__device__ __forceinline__ const T* at(const View& w, int b, int64_t t, int h) {
    return static_cast<const T*>(w.p) + b * w.sb + t * w.st + h * w.sh;
}
template <typename T>
__device__ __forceinline__ T* at_out(const View& w, int b, int64_t t, int h) {
    return static_cast<T*>(w.p) + b * w.sb + t * w.st + h * w.sh;
}

template <typename T>
__device__ __forceinline__ float dot(const float* x, const T* y, int d) {
    float s = 0.f;
    for (int c = 0; c < d; ++c) s = fmaf(x[c], to_f<T>(y[c]), s);
    return s;
}

// x_ij: score of query i (coordinates in q) and key j, base 2
template <typename T>
__device__ __forceinline__ float score2(const Args& a, float qk, int h, int64_t rel) {
    float x = qk * a.scale2;
    if (a.table != nullptr)
        x += bias2(to_f<T>(static_cast<const T*>(a.table)[h * a.table_stride + bucket_of(a, rel)]));
    return x;
}

template <typename T>
__global__ void __launch_bounds__(kT) k_forward(Args a) {
    __shared__ float q[kT], p[kT], red[4];
    const int i = (int)(blockIdx.x % a.n);
    const int h = (int)(blockIdx.x / a.n % a.H);
    const int b = (int)(blockIdx.x / a.n / a.H);
    const int t = threadIdx.x;
    if (t < a.d) q[t] = to_f<T>(at<T>(a.q, b, i, h)[t]);
    __syncthreads();
    const int end = key_end(a, b);
    const int64_t pos = (a.q_pos ? a.q_pos[b] : 0) + (int64_t)i;
    float top = -INFINITY, sum = 0.f, acc = 0.f;
    for (int j0 = 0; j0 < end; j0 += kT) {
        const int j = j0 + t;
        float x = -INFINITY;
        if (key_counts(a, b, j, end))
            x = score2<T>(a, dot<T>(q, at<T>(a.k, b, j, h / a.R), a.d), h, j - pos);
        const float mx = fmaxf(top, block_max(x, red));
        const float use = mx == -INFINITY ? 0.f : mx;
        const float alpha = ex2(top - use), e = ex2(x - use);
        sum = sum * alpha + block_sum(e, red);
        p[t] = e;
        __syncthreads();
        acc *= alpha;
        if (t < a.d)
            for (int c = 0; c < kT && j0 + c < end; ++c)
                if (p[c] != 0.f) acc = fmaf(p[c], to_f<T>(at<T>(a.v, b, j0 + c, h / a.R)[t]), acc);
        top = mx;
    }
    if (t < a.d) at_out<T>(a.o, b, i, h)[t] = from_f<T>(sum == 0.f ? 0.f : acc / sum);
    if (t == 0)
        a.lse[((int64_t)b * a.H + h) * a.n + i] = sum == 0.f ? -INFINITY : (top + lg2(sum)) * (float)kLn2;
}

// dq of one query row, delta_i, and the row's sums of ds by bucket
template <typename T>
__global__ void __launch_bounds__(kT) k_grad_q(Args a) {
    __shared__ float q[kT], g[kT], ds[kT], red[4];
    __shared__ int bu[kT];
    __shared__ float hist[kMaxBuckets];
    const int i = (int)(blockIdx.x % a.n);
    const int h = (int)(blockIdx.x / a.n % a.H);
    const int b = (int)(blockIdx.x / a.n / a.H);
    const int t = threadIdx.x;
    const int64_t row = ((int64_t)b * a.H + h) * a.n + i;
    float prod = 0.f;
    if (t < a.d) {
        q[t] = to_f<T>(at<T>(a.q, b, i, h)[t]);
        g[t] = to_f<T>(at<T>(a.dout, b, i, h)[t]);
        prod = g[t] * to_f<T>(at<T>(a.o, b, i, h)[t]);
    }
    for (int u = t; u < a.nb; u += kT) hist[u] = 0.f;
    const float delta = block_sum(prod, red);
    const float lse2 = a.lse[row] * (float)kLog2e;
    const int end = lse2 == -INFINITY ? 0 : key_end(a, b);
    const int64_t pos = (a.q_pos ? a.q_pos[b] : 0) + (int64_t)i;
    float acc = 0.f;
    for (int j0 = 0; j0 < end; j0 += kT) {
        const int j = j0 + t;
        float w = 0.f;
        __syncthreads();
        if (key_counts(a, b, j, end)) {
            const float x = score2<T>(a, dot<T>(q, at<T>(a.k, b, j, h / a.R), a.d), h, j - pos);
            w = ex2(x - lse2) * (dot<T>(g, at<T>(a.v, b, j, h / a.R), a.d) - delta);
        }
        ds[t] = w;
        if (a.bias_part) bu[t] = bucket_of(a, j - pos);
        __syncthreads();
        if (t < a.d)
            for (int c = 0; c < kT && j0 + c < end; ++c)
                if (ds[c] != 0.f) acc = fmaf(ds[c], to_f<T>(at<T>(a.k, b, j0 + c, h / a.R)[t]), acc);
        if (a.bias_part)
            for (int u = t; u < a.nb; u += kT)
                for (int c = 0; c < kT; ++c)
                    if (bu[c] == u) hist[u] += ds[c];
    }
    if (t < a.d) at_out<T>(a.dq, b, i, h)[t] = from_f<T>(acc * a.scale);
    if (t == 0) a.delta[row] = delta;
    if (a.bias_part)
        for (int u = t; u < a.nb; u += kT) a.bias_part[row * a.nb + u] = hist[u];
}

template <typename T>
__global__ void __launch_bounds__(kT) k_grad_kv(Args a) {
    __shared__ float k[kT], v[kT], p[kT], ds[kT];
    const int j = (int)(blockIdx.x % a.m);
    const int g = (int)(blockIdx.x / a.m % a.G);
    const int b = (int)(blockIdx.x / a.m / a.G);
    const int t = threadIdx.x;
    const bool counts = key_counts(a, b, j, key_end(a, b));
    if (t < a.d) {
        k[t] = to_f<T>(at<T>(a.k, b, j, g)[t]);
        v[t] = to_f<T>(at<T>(a.v, b, j, g)[t]);
    }
    float dk = 0.f, dv = 0.f;
    for (int r = 0; counts && r < a.R; ++r) {
        const int h = g * a.R + r;
        for (int i0 = 0; i0 < a.n; i0 += kT) {
            const int i = i0 + t;
            float pi = 0.f, w = 0.f;
            __syncthreads();
            if (i < a.n) {
                const int64_t row = ((int64_t)b * a.H + h) * a.n + i;
                const float lse2 = a.lse[row] * (float)kLog2e;
                if (lse2 != -INFINITY) {
                    const int64_t pos = (a.q_pos ? a.q_pos[b] : 0) + (int64_t)i;
                    const float x = score2<T>(a, dot<T>(k, at<T>(a.q, b, i, h), a.d), h, j - pos);
                    pi = ex2(x - lse2);
                    w = pi * (dot<T>(v, at<T>(a.dout, b, i, h), a.d) - a.delta[row]);
                }
            }
            p[t] = pi;
            ds[t] = w;
            __syncthreads();
            if (t < a.d)
                for (int c = 0; c < kT && i0 + c < a.n; ++c) {
                    dv = fmaf(p[c], to_f<T>(at<T>(a.dout, b, i0 + c, h)[t]), dv);
                    dk = fmaf(ds[c], to_f<T>(at<T>(a.q, b, i0 + c, h)[t]), dk);
                }
        }
    }
    if (t < a.d) {
        at_out<T>(a.dk, b, j, g)[t] = from_f<T>(dk * a.scale);
        at_out<T>(a.dv, b, j, g)[t] = from_f<T>(dv);
    }
}

// dbias[h][u] over batches and rows (and heads, for a shared row), in order
template <typename T>
__global__ void __launch_bounds__(kT) k_grad_bias(Args a, T* __restrict__ dbias) {
    __shared__ float red[4];
    const int u = blockIdx.x % a.nb;
    const int hb = blockIdx.x / a.nb;
    const int h0 = a.table_stride ? hb : 0, h1 = a.table_stride ? hb + 1 : a.H;
    float s = 0.f;
    for (int b = 0; b < a.B; ++b)
        for (int h = h0; h < h1; ++h)
            for (int i = threadIdx.x; i < a.n; i += kT)
                s += a.bias_part[(((int64_t)b * a.H + h) * a.n + i) * a.nb + u];
    s = block_sum(s, red);
    if (threadIdx.x == 0) dbias[blockIdx.x] = from_f<T>(s);
}

template <typename T>
cudaError_t grad_simple(const Args& a, void* dbias, cudaStream_t s) {
    const int64_t rows = (int64_t)a.B * a.H * a.n, keys = (int64_t)a.B * a.G * a.m;
    if (rows) {
        k_grad_q<T><<<(unsigned)rows, kT, 0, s>>>(a);
        count_launch();
    }
    if (keys) {
        k_grad_kv<T><<<(unsigned)keys, kT, 0, s>>>(a);
        count_launch();
    }
    if (dbias) {
        k_grad_bias<T><<<(unsigned)((a.table_stride ? a.H : 1) * a.nb), kT, 0, s>>>(
            a, static_cast<T*>(dbias));
        count_launch();
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_forward_simple(const Args& a, cudaStream_t s) {
    const unsigned rows = (unsigned)((int64_t)a.B * a.H * a.n);
    if (a.bf16)
        k_forward<__nv_bfloat16><<<rows, kT, 0, s>>>(a);
    else
        k_forward<__half><<<rows, kT, 0, s>>>(a);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_grad_simple(const Args& a, void* dbias, cudaStream_t s) {
    return a.bf16 ? grad_simple<__nv_bfloat16>(a, dbias, s) : grad_simple<__half>(a, dbias, s);
}

}  // namespace attn
}  // namespace fs
