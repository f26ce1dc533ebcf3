// C ABI of cross attention: argument checks, workspace, choice of kernels.
#include "fs_attn_host.cuh"

#include <algorithm>
#include <cmath>

namespace fs {
namespace attn {

// -1 without one (every pointer then fails its check)
int current_device() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError();
    return dev;
}

// a device array of device dev, the current one (empty tensors may be null)
fs_status check_ptr(int dev, const void* p, int64_t count, const char* name) {
    if (count == 0) return FS_OK;
    if (!p) return fail(FS_ERR_INVALID_ARG, "null %s", name);
    cudaPointerAttributes attr;
    if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
        cudaGetLastError();
        return fail(FS_ERR_INVALID_ARG, "%s: unknown pointer", name);
    }
    if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged)
        return fail(FS_ERR_INVALID_ARG, "%s must be device memory", name);
    if (attr.type == cudaMemoryTypeDevice && attr.device != dev)
        return fail(FS_ERR_INVALID_ARG, "%s on device %d, current is %d", name, attr.device, dev);
    return FS_OK;
}

fs_status view(int dev, View& w, const void* p, const int64_t* stride, int64_t batch, int64_t tokens,
               int heads, int d, bool out, const char* name) {
    FS_TRY(check_ptr(dev, p, batch * tokens, name));
    w.p = const_cast<void*>(p);
    w.sb = stride[0];
    w.st = stride[1];
    w.sh = stride[2];
    for (int i = 0; i < 3; ++i)
        if (stride[i] < 0) return fail(FS_ERR_INVALID_ARG, "%s has a negative stride", name);
    if (!out || batch == 0 || tokens == 0) return FS_OK;
    // A result's axes by rising stride: each steps over all that the ones before it span.
    struct Axis {
        int64_t size, stride;
    } axis[3] = {{batch, stride[0]}, {tokens, stride[1]}, {heads, stride[2]}};
    std::sort(axis, axis + 3, [](const Axis& x, const Axis& y) { return x.stride < y.stride; });
    double span = d;        // (products of two sizes may pass 64 bits)
    for (const Axis& x : axis) {
        if (x.size == 1) continue;
        if ((double)x.stride < span) return fail(FS_ERR_INVALID_ARG, "the rows of %s overlap", name);
        span += (double)x.stride * (double)(x.size - 1);
    }
    return FS_OK;
}

bool aligned16(const View& w, int B, int tokens, int heads) {
    return (reinterpret_cast<uintptr_t>(w.p) & 15) == 0 && (tokens <= 1 || w.st % 8 == 0) &&
           (heads <= 1 || w.sh % 8 == 0) && (B <= 1 || w.sb % 8 == 0);
}

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
    if (!(a->scale > 0.f) || !std::isfinite((float)(a->scale * kLog2e)))
        return fail(FS_ERR_INVALID_ARG, "scale must be positive and finite in base 2 (got %g)",
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

fs_status fill(int dev, Args& w, const fs_attention* a) {
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
    FS_TRY(check_ptr(dev, a->kv_len, a->kv_len ? a->batch : 0, "kv_len"));
    FS_TRY(check_ptr(dev, a->key_mask, a->key_mask ? a->batch * a->m : 0, "key_mask"));
    FS_TRY(check_ptr(dev, a->q_pos, a->q_pos ? a->batch : 0, "q_pos"));
    w.kv_len = a->kv_len;
    w.mask = a->key_mask;
    w.mask_stride = a->mask_stride;
    if (a->n_buckets) {
        FS_TRY(check_ptr(dev, a->bias, 1, "bias"));
        FS_TRY(check_ptr(dev, a->bias_buckets, 1, "bias_buckets"));
        w.table = a->bias;
        w.table_stride = a->bias_stride;
        w.buckets = a->bias_buckets;
        w.nb = a->n_buckets;
        w.D = a->max_distance;
        w.q_pos = a->q_pos;
    }
    return FS_OK;
}

fs_status check_rows(double rows) {
    if (rows > (double)INT32_MAX)
        return fail(FS_ERR_UNSUPPORTED, "%.3g rows of queries or keys in one call", rows);
    return FS_OK;
}

// What a tensor map can describe: 16-byte steps, below 2^40 bytes, and tokens
// that differ.
bool mappable(const View& w, int B, int tokens, int heads, int d) {
    constexpr int64_t far = int64_t(1) << 39;
    return d % 8 == 0 && aligned16(w, B, tokens, heads) && (tokens <= 1 || w.st > 0) && w.st < far &&
           w.sh < far && w.sb < far;
}

// An input that the kernels read through a tensor map (or 16 bytes at a time):
// in place, or from a copy in the workspace with rows of 16-byte multiples.
struct Input {
    View* w;
    int tokens, heads;
    bool copy = false;
    size_t off = 0;
    Input(View& v, int t, int h) : w(&v), tokens(t), heads(h) {}
    void plan(const Args& a, Layout& L, bool map = true) {
        copy = map ? !mappable(*w, a.B, tokens, heads, a.d)
                   : a.d % 8 != 0 || !aligned16(*w, a.B, tokens, heads);
        if (copy) off = L.take(2 * (size_t)a.B * tokens * heads * pitch(a));
    }
    static int pitch(const Args& a) { return (a.d + 7) / 8 * 8; }
    fs_status run(const Call& c, const Args& a) {
        if (!copy) return FS_OK;
        const int dp = pitch(a);
        void* to = c.at<void>(off);
        FS_CUDA(launch_pack(*w, to, a.B, tokens, heads, a.d, dp, c.stream));
        w->p = to;
        w->sh = dp;
        w->st = (int64_t)heads * dp;
        w->sb = (int64_t)tokens * heads * dp;
        return FS_OK;
    }
};

// The key tiles of a mask.
struct TilePlan {
    KeyTiles kt = {};
    size_t words = 0, list = 0, count = 0;
    void plan(const Args& a, Layout& L) {
        kt.tiles = (a.m + kTile - 1) / kTile;
        if (!a.mask) return;
        words = L.take(sizeof(uint4) * (size_t)a.B * kt.tiles);
        list = L.take(sizeof(int) * (size_t)a.B * kt.tiles);
        count = L.take(sizeof(int) * (size_t)a.B);
    }
    fs_status run(const Call& c, const Args& a) {
        if (!a.mask) return FS_OK;
        kt.words = c.at<uint4>(words);
        kt.list = c.at<int>(list);
        kt.count = c.at<int>(count);
        FS_CUDA(launch_key_tiles(a, c.at<uint4>(words), c.at<int>(list), c.at<int>(count), kt.tiles,
                                 c.stream));
        return FS_OK;
    }
};

// Splits of the keys: enough blocks for every SM, of two key tiles at least.
int choose_key_splits(int64_t blocks, int tiles, int sms) {
    int64_t s = blocks >= sms ? 1 : sms / blocks;
    s = std::min<int64_t>(s, (tiles + 1) / 2);
    return (int)std::max<int64_t>(s, 1);
}

// Key tiles up to which delta comes from the scores without a bias gradient too: the fewer
// keys share a row's weight, the more the rounding of O counts.  In bfloat16 dq is 0.28 %
// off with delta from O at 150 to 830 keys, 0.25 % at 4096; with it from the scores 0.24 %
// (3 x 2644 queries, 478 keys, 16 heads on 8 of 32, forward and gradients: 169 us for 128).
constexpr int kExactTiles = 8;

// Splits of the gradients' tiles, at most so: as many as a block's tiles outlast the whole
// call's when those are spread evenly (a block's fixed part counts as 2.5 of them).  Where
// k_grad_delta, of the queries' blocks alone, comes first, their number counts alone.
// 2 x 60 queries, 6171 keys, 16 heads on 8 of 112: 93 us for 102, with a bias 153 for
// 234; 3230 queries, 140 keys, 2 heads on 1 of 128, bias: 72 for 99; 4 x 351 queries, 157
// keys, 64 heads on 8 of 64 (64 blocks of keys beside 768 of queries): 123 us, and 143 with
// the keys' blocks split.
void choose_grad_splits(GradArgs& p, int sms) {
    const Args& a = p.a;
    const int64_t q_blocks = (int64_t)p.q_tiles * a.H * a.B, k_blocks = (int64_t)p.k_tiles * a.G * a.B;
    const int q_steps = p.k_tiles, k_steps = a.R * p.q_tiles;
    const double even = (q_blocks * (q_steps + 2.5) + k_blocks * (k_steps + 2.5)) / sms;
    p.q_splits = choose_key_splits(q_blocks, q_steps, sms);
    p.k_splits = choose_key_splits(k_blocks, k_steps, sms);
    if (!p.exact_delta) p.q_splits = std::min(p.q_splits, (int)std::ceil(q_steps / even));
    p.k_splits = std::min(p.k_splits, (int)std::ceil(k_steps / even));
}

// Whether the few-query kernel takes a call: one tile of its 16 rows per key head, or
// two where query heads share keys (the 128-row tiles of the other kernel then read
// the keys once per query head; with a head of its own each they read them once
// too).  8 heads of 64, 21 queries and 77 keys: 8.0 us here, 7.0 us there; 4 queries
// of 8 heads to a key head, 20000 keys: twice as fast here.
bool few_rows(const Args& a) {
    const int64_t rows = (int64_t)a.R * a.n;
    return rows <= 16 || (rows <= 32 && a.R > 1);
}

// Its splits of the keys.  A split costs its keys and a fixed part (set-up, its share
// of the join) worth about 512 keys; blocks beyond the resident ones wait for a
// whole turn.  The fewest splits of the least cost.
int choose_decode_splits(int64_t blocks, int m, int64_t resident) {
    constexpr double kFixedKeys = 512.0;
    if (blocks > kCounters) return 1;
    const int64_t most = std::min<int64_t>((m + kDecodeKeys - 1) / kDecodeKeys, 4 * resident / blocks + 1);
    int best = 1;
    double least = 0.0;
    for (int64_t s = 1; s <= most; ++s) {
        const double turns = (double)((blocks * s + resident - 1) / resident);
        const double cost = turns * ((double)m / (double)s + kFixedKeys);
        if (s == 1 || cost < 0.999 * least) {
            least = cost;
            best = (int)s;
        }
    }
    return best;
}

fs_status forward_entry(const fs_attention* at, const void* q, const void* k, const void* v,
                        void* out, float* lse, void* stream) {
    FS_TRY(check_desc(at));
    FwdArgs p = {};
    Args& a = p.a;
    const int dev = current_device();
    FS_TRY(fill(dev, a, at));
    FS_TRY(view(dev, a.q, q, at->q_stride, at->batch, at->n, a.H, a.d, false, "q"));
    FS_TRY(view(dev, a.k, k, at->k_stride, at->batch, at->m, a.G, a.d, false, "k"));
    FS_TRY(view(dev, a.v, v, at->v_stride, at->batch, at->m, a.G, a.d, false, "v"));
    FS_TRY(view(dev, a.o, out, at->out_stride, at->batch, at->n, a.H, a.d, true, "out"));
    FS_TRY(check_ptr(dev, lse, at->batch * at->n, "lse"));
    a.lse = lse;
    FS_TRY(check_rows((double)at->batch * a.H * at->n));
    FS_TRY(check_rows((double)at->batch * a.G * at->m));
    const int64_t rows = at->batch * a.H * at->n;
    if (rows == 0) return FS_OK;
    NvtxRange range("fs_cross_attention");
    Call c;
    if (a.m == 0) {
        FS_TRY(begin_call(c, stream, false));
        FS_CUDA(launch_zero(a, a.o, a.n, a.H, lse, c.stream));
        return FS_OK;
    }
    int sms = 0;
    FS_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    Input inputs[3] = {{a.q, a.n, a.H}, {a.k, a.m, a.G}, {a.v, a.m, a.G}};
    const bool few = few_rows(a);
    for (Input& x : inputs) x.plan(a, c.L, !few);
    TilePlan tiles;
    DecodeArgs dp = {};
    int splits;
    if (few) {
        dp.row_blocks = a.R * a.n <= 8 ? 1 : 2;
        dp.groups = (a.R * a.n + 8 * dp.row_blocks - 1) / (8 * dp.row_blocks);
        dp.dp = (a.d + 3) / 4 * 4;
        int resident = 0;
        FS_CUDA(decode_resident(a, dp.row_blocks, &resident));
        splits = choose_decode_splits((int64_t)a.B * a.G * dp.groups, a.m, (int64_t)sms * resident);
    } else {
        tiles.plan(a, c.L);
        p.row_blocks = (a.n + 2 * kTile - 1) / (2 * kTile);
        splits = choose_key_splits((int64_t)p.row_blocks * a.H * a.B, tiles.kt.tiles, sms);
    }
    Partials part = {};
    part.rows = rows;
    size_t part_out = 0, part_lse = 0;
    if (splits > 1) {
        part_out = c.L.take(sizeof(float) * (size_t)splits * rows * ((a.d + 3) / 4 * 4));
        part_lse = c.L.take(sizeof(float) * (size_t)splits * rows);
    }
    const bool scratch = c.L.off > 0;
    FS_TRY(begin_call(c, stream, scratch));
    FS_TRY(ensure_capacity(c));
    for (Input& x : inputs) FS_TRY(x.run(c, a));
    if (splits > 1) {
        part.out = c.at<float>(part_out);
        part.lse2 = c.at<float>(part_lse);
    }
    a.err = c.ws->err_word;
    if (few) {
        dp.a = a;
        dp.part = part;
        dp.splits = splits;
        dp.counters = c.ws->counters;
        FS_CUDA(launch_decode(dp, c.stream));
        return scratch ? end_call(c) : FS_OK;
    }
    FS_TRY(tiles.run(c, a));
    p.kt = tiles.kt;
    p.part = part;
    p.splits = splits;
    p.out_vec = a.d % 8 == 0 && aligned16(a.o, a.B, a.n, a.H);
    FS_TRY(make_tensor_map(p.q, a.q, a.B, a.n, a.H, a.d, a.bf16));
    FS_TRY(make_tensor_map(p.k, a.k, a.B, a.m, a.G, a.d, a.bf16, forward_keys(a.d)));
    FS_TRY(make_tensor_map(p.v, a.v, a.B, a.m, a.G, a.d, a.bf16, forward_keys(a.d)));
    FS_CUDA(launch_forward_tc(p, c.stream));
    if (splits > 1) FS_CUDA(launch_combine(a, part, splits, c.stream));
    return scratch ? end_call(c) : FS_OK;
}

fs_status grad_entry(const fs_attention* at, const void* q, const void* k, const void* v,
                     const void* out, const float* lse, const void* dout, void* dq, void* dk,
                     void* dv, void* dbias, void* stream) {
    FS_TRY(check_desc(at));
    GradArgs p = {};
    Args& a = p.a;
    const int dev = current_device();
    FS_TRY(fill(dev, a, at));
    FS_TRY(view(dev, a.q, q, at->q_stride, at->batch, at->n, a.H, a.d, false, "q"));
    FS_TRY(view(dev, a.k, k, at->k_stride, at->batch, at->m, a.G, a.d, false, "k"));
    FS_TRY(view(dev, a.v, v, at->v_stride, at->batch, at->m, a.G, a.d, false, "v"));
    FS_TRY(view(dev, a.o, out, at->out_stride, at->batch, at->n, a.H, a.d, false, "out"));
    FS_TRY(view(dev, a.dout, dout, at->dout_stride, at->batch, at->n, a.H, a.d, false, "dout"));
    FS_TRY(view(dev, a.dq, dq, at->dq_stride, at->batch, at->n, a.H, a.d, true, "dq"));
    FS_TRY(view(dev, a.dk, dk, at->dk_stride, at->batch, at->m, a.G, a.d, true, "dk"));
    FS_TRY(view(dev, a.dv, dv, at->dv_stride, at->batch, at->m, a.G, a.d, true, "dv"));
    FS_TRY(check_ptr(dev, lse, at->batch * at->n, "lse"));
    if (dbias && !at->n_buckets) return fail(FS_ERR_INVALID_ARG, "dbias without a bias");
    if (dbias) FS_TRY(check_ptr(dev, dbias, 1, "dbias"));
    a.lse = const_cast<float*>(lse);
    FS_TRY(check_rows((double)at->batch * a.H * at->n));
    FS_TRY(check_rows((double)at->batch * a.G * at->m));
    NvtxRange range("fs_cross_attention_grad");
    Call c;
    if (a.n == 0 || a.m == 0 || a.B == 0) {
        FS_TRY(begin_call(c, stream, false));
        FS_CUDA(launch_zero(a, a.dq, a.n, a.H, nullptr, c.stream));
        FS_CUDA(launch_zero(a, a.dk, a.m, a.G, nullptr, c.stream));
        FS_CUDA(launch_zero(a, a.dv, a.m, a.G, nullptr, c.stream));
        if (dbias)
            FS_CUDA(cudaMemsetAsync(dbias, 0, 2 * (size_t)(a.table_stride ? a.H : 1) * a.nb, c.stream));
        return FS_OK;
    }
    Input inputs[4] = {{a.q, a.n, a.H}, {a.k, a.m, a.G}, {a.v, a.m, a.G}, {a.dout, a.n, a.H}};
    TilePlan tiles;
    for (Input& x : inputs) x.plan(a, c.L);
    tiles.plan(a, c.L);
    p.q_tiles = (a.n + kTile - 1) / kTile;
    p.k_tiles = tiles.kt.tiles;
    const size_t blocks = (size_t)a.B * a.H * p.q_tiles;
    int sms = 0;
    FS_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    p.exact_delta = dbias || p.k_tiles <= kExactTiles;
    choose_grad_splits(p, sms);
    const size_t rows = c.L.take(blocks * kRowStride);
    const size_t part = c.L.take(dbias ? sizeof(float) * blocks * p.q_splits * (2 * (size_t)a.D + 1) : 0);
    const size_t q_part = p.q_splits > 1 ? sizeof(float) * p.q_splits : 0;
    const size_t k_part = p.k_splits > 1 ? sizeof(float) * p.k_splits * a.B * a.G * a.m * a.d : 0;
    const size_t part_dq = c.L.take(q_part * a.B * a.H * a.n * a.d);
    const size_t part_delta = c.L.take(p.exact_delta ? q_part * blocks * kTile : 0);
    const size_t part_dk = c.L.take(k_part), part_dv = c.L.take(k_part);
    const size_t entry = a.bf16 ? 0 : sizeof(float);
    const size_t q_range = c.L.take(entry * blocks * 4);
    const size_t v_range = c.L.take(p.exact_delta ? 0 : entry * a.B * a.G * p.k_tiles);
    const size_t part_top = c.L.take(p.exact_delta && p.q_splits > 1 ? entry * p.q_splits * blocks * kTile : 0);
    FS_TRY(begin_call(c, stream));
    FS_TRY(ensure_capacity(c));
    for (Input& x : inputs) FS_TRY(x.run(c, a));
    FS_TRY(tiles.run(c, a));
    p.kt = tiles.kt;
    p.rows = c.at<uint8_t>(rows);
    a.bias_part = dbias ? c.at<float>(part) : nullptr;
    p.part_dq = c.at<float>(part_dq);
    p.part_delta = c.at<float>(part_delta);
    p.part_dk = c.at<float>(part_dk);
    p.part_dv = c.at<float>(part_dv);
    p.q_range = c.at<float>(q_range);
    p.v_range = c.at<float>(v_range);
    p.part_top = c.at<float>(part_top);
    a.err = c.ws->err_word;
    auto vec = [&](const View& w, int tokens, int heads) {
        return a.d % 8 == 0 && aligned16(w, a.B, tokens, heads);
    };
    p.dout_vec = vec(a.dout, a.n, a.H);
    p.o_vec = vec(a.o, a.n, a.H);
    p.dq_vec = vec(a.dq, a.n, a.H);
    p.dk_vec = vec(a.dk, a.m, a.G);
    p.dv_vec = vec(a.dv, a.m, a.G);
    FS_TRY(make_tensor_map(p.q, a.q, a.B, a.n, a.H, a.d, a.bf16));
    FS_TRY(make_tensor_map(p.k, a.k, a.B, a.m, a.G, a.d, a.bf16));
    FS_TRY(make_tensor_map(p.v, a.v, a.B, a.m, a.G, a.d, a.bf16));
    FS_TRY(make_tensor_map(p.dout, a.dout, a.B, a.n, a.H, a.d, a.bf16));
    FS_CUDA(launch_grad_tc(p, dbias, c.stream));
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
