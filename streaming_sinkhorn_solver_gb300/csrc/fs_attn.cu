// C ABI of cross attention: argument checks, workspace, choice of kernels.
#include "fs_host.cuh"
#include "fs_attn.cuh"

#include <cmath>

namespace fs {
namespace attn {

namespace {

fs_status check_desc(const fs_attention* a) {
    if (!a) return fail(FS_ERR_INVALID_ARG, "null fs_attention");
    if (a->dtype != FS_DTYPE_BF16 && a->dtype != FS_DTYPE_F16)
        return fail(FS_ERR_INVALID_ARG, "fs_attention.dtype=%d", a->dtype);
    if (a->heads < 1 || a->kv_heads < 1 || a->heads % a->kv_heads != 0)
        return fail(FS_ERR_INVALID_ARG, "heads=%d is not a multiple of kv_heads=%d", a->heads,
                    a->kv_heads);
    if (a->d < 1 || a->d > kMaxHeadDim)
        return fail(FS_ERR_INVALID_ARG, "d=%d out of range [1, %d]", a->d, kMaxHeadDim);
    constexpr int64_t kMaxTokens = INT32_MAX - 4096;   // tile ends stay in 32 bits
    if (a->batch < 0 || a->n < 0 || a->m < 0 || a->batch > kMaxTokens || a->n > kMaxTokens ||
        a->m > kMaxTokens)
        return fail(FS_ERR_INVALID_ARG, "batch=%lld n=%lld m=%lld out of range [0, %lld]",
                    (long long)a->batch, (long long)a->n, (long long)a->m, (long long)kMaxTokens);
    if (!(a->scale > 0.f) || !std::isfinite(a->scale))
        return fail(FS_ERR_INVALID_ARG, "scale must be positive and finite (got %g)",
                    (double)a->scale);
    if (a->reserved) return fail(FS_ERR_INVALID_ARG, "fs_attention.reserved must be zero");
    if (a->n_buckets < 0 || a->n_buckets > kMaxBuckets)
        return fail(FS_ERR_INVALID_ARG, "n_buckets=%d out of range [0, %d]", a->n_buckets,
                    kMaxBuckets);
    if (a->n_buckets) {
        if (!a->bias || !a->bias_buckets) return fail(FS_ERR_INVALID_ARG, "null bias or bias_buckets");
        if (a->max_distance < 1 || a->max_distance > kMaxDistance)
            return fail(FS_ERR_INVALID_ARG, "max_distance=%d out of range [1, %d]", a->max_distance,
                        kMaxDistance);
        if (a->bias_stride != 0 && a->bias_stride < a->n_buckets)
            return fail(FS_ERR_INVALID_ARG, "bias_stride=%lld is less than n_buckets=%d",
                        (long long)a->bias_stride, a->n_buckets);
    }
    if (a->key_mask && a->mask_stride < 0) return fail(FS_ERR_INVALID_ARG, "negative mask_stride");
    return FS_OK;
}

// a device array of the current device (empty tensors may be null)
fs_status check_ptr(const void* p, int64_t count, const char* name) {
    if (count == 0) return FS_OK;
    if (!p) return fail(FS_ERR_INVALID_ARG, "null %s", name);
    cudaPointerAttributes attr;
    if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
        cudaGetLastError();
        return fail(FS_ERR_INVALID_ARG, "%s: unknown pointer", name);
    }
    if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged)
        return fail(FS_ERR_INVALID_ARG, "%s must be device memory", name);
    return FS_OK;
}

fs_status view(View& w, const void* p, const int64_t* stride, int64_t batch, int64_t tokens,
               int heads, int d, bool out, const char* name) {
    FS_TRY(check_ptr(p, batch * tokens, name));
    w.p = const_cast<void*>(p);
    w.sb = stride[0];
    w.st = stride[1];
    w.sh = stride[2];
    const int64_t size[3] = {batch, tokens, heads};
    for (int i = 0; i < 3; ++i) {
        if (stride[i] < 0) return fail(FS_ERR_INVALID_ARG, "%s has a negative stride", name);
        if (out && size[i] > 1 && stride[i] < d)
            return fail(FS_ERR_INVALID_ARG, "the rows of %s overlap", name);
    }
    return FS_OK;
}

fs_status fill(Args& w, const fs_attention* a) {
    w.B = (int)a->batch;
    w.H = a->heads;
    w.G = a->kv_heads;
    w.R = a->heads / a->kv_heads;
    w.n = (int)a->n;
    w.m = (int)a->m;
    w.d = a->d;
    w.bf16 = a->dtype == FS_DTYPE_BF16;
    w.scale = a->scale;
    w.scale2 = (float)((double)a->scale * kLog2e);
    FS_TRY(check_ptr(a->kv_len, a->kv_len ? a->batch : 0, "kv_len"));
    FS_TRY(check_ptr(a->key_mask, a->key_mask ? a->batch * a->m : 0, "key_mask"));
    FS_TRY(check_ptr(a->q_pos, a->q_pos ? a->batch : 0, "q_pos"));
    w.kv_len = a->kv_len;
    w.mask = a->key_mask;
    w.mask_stride = a->mask_stride;
    if (a->n_buckets) {
        FS_TRY(check_ptr(a->bias, 1, "bias"));
        FS_TRY(check_ptr(a->bias_buckets, 1, "bias_buckets"));
        w.table = a->bias;
        w.table_stride = a->bias_stride;
        w.buckets = a->bias_buckets;
        w.nb = a->n_buckets;
        w.D = a->max_distance;
        w.q_pos = a->q_pos;
    }
    return FS_OK;
}

fs_status check_tiles(double tiles) {
    if (tiles > (double)INT32_MAX)
        return fail(FS_ERR_UNSUPPORTED, "%.3g tiles of work in one call", tiles);
    return FS_OK;
}

fs_status forward_entry(const fs_attention* at, const void* q, const void* k, const void* v,
                        void* out, float* lse, void* stream) {
    FS_TRY(check_desc(at));
    Args a = {};
    FS_TRY(fill(a, at));
    FS_TRY(view(a.q, q, at->q_stride, at->batch, at->n, a.H, a.d, false, "q"));
    FS_TRY(view(a.k, k, at->k_stride, at->batch, at->m, a.G, a.d, false, "k"));
    FS_TRY(view(a.v, v, at->v_stride, at->batch, at->m, a.G, a.d, false, "v"));
    FS_TRY(view(a.o, out, at->out_stride, at->batch, at->n, a.H, a.d, true, "out"));
    FS_TRY(check_ptr(lse, at->batch * at->n, "lse"));
    a.lse = lse;
    FS_TRY(check_tiles((double)at->batch * a.H * at->n));
    const int64_t rows = at->batch * a.H * at->n;
    if (rows == 0) return FS_OK;
    NvtxRange range("fs_cross_attention");
    FS_CUDA(launch_forward_simple(a, static_cast<cudaStream_t>(stream)));
    return FS_OK;
}

fs_status grad_entry(const fs_attention* at, const void* q, const void* k, const void* v,
                     const void* out, const float* lse, const void* dout, void* dq, void* dk,
                     void* dv, void* dbias, void* stream) {
    FS_TRY(check_desc(at));
    Args a = {};
    FS_TRY(fill(a, at));
    FS_TRY(view(a.q, q, at->q_stride, at->batch, at->n, a.H, a.d, false, "q"));
    FS_TRY(view(a.k, k, at->k_stride, at->batch, at->m, a.G, a.d, false, "k"));
    FS_TRY(view(a.v, v, at->v_stride, at->batch, at->m, a.G, a.d, false, "v"));
    FS_TRY(view(a.o, out, at->out_stride, at->batch, at->n, a.H, a.d, false, "out"));
    FS_TRY(view(a.dout, dout, at->dout_stride, at->batch, at->n, a.H, a.d, false, "dout"));
    FS_TRY(view(a.dq, dq, at->dq_stride, at->batch, at->n, a.H, a.d, true, "dq"));
    FS_TRY(view(a.dk, dk, at->dk_stride, at->batch, at->m, a.G, a.d, true, "dk"));
    FS_TRY(view(a.dv, dv, at->dv_stride, at->batch, at->m, a.G, a.d, true, "dv"));
    FS_TRY(check_ptr(lse, at->batch * at->n, "lse"));
    if (dbias && !at->n_buckets) return fail(FS_ERR_INVALID_ARG, "dbias without a bias");
    if (dbias) FS_TRY(check_ptr(dbias, 1, "dbias"));
    a.lse = const_cast<float*>(lse);
    FS_TRY(check_tiles((double)at->batch * a.H * at->n));
    const int64_t rows = at->batch * a.H * at->n;
    FS_TRY(check_tiles((double)at->batch * a.G * at->m));
    NvtxRange range("fs_cross_attention_grad");
    Call c;
    FS_TRY(begin_call(c, stream));
    const size_t o_delta = c.L.take(sizeof(float) * (size_t)rows);
    const size_t o_part = c.L.take(dbias ? sizeof(float) * (size_t)rows * a.nb : 0);
    FS_TRY(ensure_capacity(c));
    a.delta = c.at<float>(o_delta);
    a.bias_part = dbias ? c.at<float>(o_part) : nullptr;
    a.err = c.ws->err_word;
    FS_CUDA(launch_grad_simple(a, dbias, c.stream));
    return end_call(c);
}

}  // namespace

}  // namespace attn
}  // namespace fs

using namespace fs;

extern "C" {

fs_status fs_cross_attention(const fs_attention* at, const void* q, const void* k, const void* v,
                             void* out, float* lse, void* stream) {
    try {
        return attn::forward_entry(at, q, k, v, out, lse, stream);
    } catch (...) {
        return fail(FS_ERR_CUDA, "unexpected host exception");
    }
}

fs_status fs_cross_attention_grad(const fs_attention* at, const void* q, const void* k,
                                  const void* v, const void* out, const float* lse,
                                  const void* dout, void* dq, void* dk, void* dv, void* dbias,
                                  void* stream) {
    try {
        return attn::grad_entry(at, q, k, v, out, lse, dout, dq, dk, dv, dbias, stream);
    } catch (...) {
        return fail(FS_ERR_CUDA, "unexpected host exception");
    }
}

}  // extern "C"
