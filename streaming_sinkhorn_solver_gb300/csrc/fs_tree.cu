// C ABI of the tree attention: argument checks, workspace, choice of kernels.
#include "fs_tree.cuh"

#include <cmath>

namespace fs {
namespace tree {

namespace {

// Splits of the keys of the few-row kernel.  A split costs its keys and a fixed part
// (set-up, its share of the join) worth about 512 keys of 16 bits, 256 of 8; blocks beyond the
// resident ones come as others end, between whole turns (sequences of one length) and none.  The
// fewest splits of the least cost.
int choose_few_splits(int64_t blocks, int m, int64_t resident, bool bytes) {
    const double fixed = bytes ? 256.0 : 512.0;
    if (blocks > kCounters) return 1;
    const int64_t most = std::min<int64_t>((m + kFewKeys - 1) / kFewKeys, 4 * resident / blocks + 1);
    int best = 1;
    double least = 0.0;
    for (int64_t s = 1; s <= most; ++s) {
        const double full = (double)(blocks * s) / (double)resident;
        const double turns = full <= 1.0 ? 1.0 : 0.5 * (std::ceil(full) + full + 0.5);
        const double cost = turns * ((double)m / (double)s + fixed);
        if (s == 1 || cost < 0.999 * least) {
            least = cost;
            best = (int)s;
        }
    }
    return best;
}

// Splits of the keys of the tensor-core kernel, one block to an SM: a split costs its tiles
// and a fixed part worth about 8 of them (set-up, its results); the join of several about
// 12.  The fewest splits of the least cost.
int choose_tc_splits(int64_t blocks, int m, int sms) {
    constexpr double kFixed = 8.0, kJoin = 12.0;
    const int tiles = (m + kTcKeys - 1) / kTcKeys;
    const int64_t most = std::min<int64_t>((tiles + 3) / 4, 4 * (int64_t)sms / blocks + 1);
    int best = 1;
    double least = 0.0;
    for (int64_t s = 1; s <= most; ++s) {
        const double turns = (double)((blocks * s + sms - 1) / sms);
        const double cost = turns * ((double)((tiles + s - 1) / s) + kFixed) + (s > 1 ? kJoin : 0.0);
        if (s == 1 || cost < 0.999 * least) {
            least = cost;
            best = (int)s;
        }
    }
    return best;
}

// Whether the few-row kernel takes a call: caches whose rows cannot be copied by the page, and up to
// one block of 8 rows to a key head, in 16 bits and heads above 64 only where there is little to read.
// The table's reach stands for the lengths, which are on the GPU.
// Measured with 4 rows on each of 8 key heads (few rows, tensor cores), us:
//   bfloat16 heads of 128: 34 MB 15, 16; 67 MB 24, 22; 134 MB 38, 30; 319 MB 71, 54; 1275 MB 240, 188
//   bfloat16 heads of 64:  34 MB 14, 15; 67 MB 22, 18; 134 MB 34, 35; 319 MB 59, 59; 1275 MB 199, 203
//   e4m3 of 128, 64, as many keys: 34 MB 14, 19 and 14, 21; 319 MB 40, 51 and 44, 82; 1275 MB 117, 172
//   and 129, 293
// (Beyond 8 rows, where a cache would be read twice: 12 rows of heads of 128, e4m3 47, 49, bfloat16 67, 55.)
bool few_rows(const Args& a) {
    constexpr double kLittle = 48e6;
    if (!tc_copies(a.c)) return true;
    if (a.R * a.n > 8) return false;
    return a.c.held != kv::HELD_16 || a.d <= 64 || 4.0 * a.c.B * a.c.G * a.c.reach() * a.d <= kLittle;
}

fs_status tree_entry(const fs_cache* cache, const fs_tree* t, const void* q, void* out, float* lse,
                     void* stream) {
    const int dev = attn::current_device();
    FewArgs p = {};
    Args& a = p.a;
    FS_TRY(kv::fill_cache(dev, a.c, cache, false));
    if (!t) return fail(FS_ERR_INVALID_ARG, "null fs_tree");
    if (t->dtype != FS_DTYPE_BF16 && t->dtype != FS_DTYPE_F16)
        return fail(FS_ERR_INVALID_ARG, "fs_tree.dtype=%d", t->dtype);
    if (cache->dtype < FS_DTYPE_E4M3 && t->dtype != cache->dtype)
        return fail(FS_ERR_INVALID_ARG, "queries of dtype %d for a cache of dtype %d", t->dtype, cache->dtype);
    constexpr int kMostHeads = 1 << 16;
    if (t->heads < 1 || t->heads > kMostHeads || t->heads % a.c.G != 0)
        return fail(FS_ERR_INVALID_ARG, "heads=%d is not a multiple of kv_heads=%d", t->heads, a.c.G);
    if (t->n < 0 || t->n > kv::kMaxTree)
        return fail(FS_ERR_INVALID_ARG, "n=%lld out of range [0, %d]", (long long)t->n, kv::kMaxTree);
    if (!(t->scale > 0.f) || !std::isfinite((float)(t->scale * kLog2e)))
        return fail(FS_ERR_INVALID_ARG, "scale must be positive and finite in base 2 (got %g)",
                    (double)t->scale);
    if (t->reserved) return fail(FS_ERR_INVALID_ARG, "fs_tree.reserved must be zero");
    if (t->parents && t->parents_stride < 0) return fail(FS_ERR_INVALID_ARG, "negative parents_stride");
    a.H = t->heads;
    a.R = t->heads / a.c.G;
    a.n = (int)t->n;
    a.d = a.c.d;
    a.bf16 = t->dtype == FS_DTYPE_BF16;
    a.scale2 = (float)((double)t->scale * kLog2e);
    const int64_t B = a.c.B;
    FS_TRY(attn::view(dev, a.q, q, t->q_stride, B, t->n, a.H, a.d, false, "q"));
    FS_TRY(attn::view(dev, a.o, out, t->out_stride, B, t->n, a.H, a.d, true, "out"));
    FS_TRY(attn::check_ptr(dev, lse, B * t->n, "lse"));
    FS_TRY(attn::check_ptr(dev, t->ctx_len, B * t->n, "ctx_len"));
    FS_TRY(attn::check_ptr(dev, t->parents, t->parents ? B * t->n : 0, "parents"));
    if ((double)B * a.H * a.n > (double)INT32_MAX)
        return fail(FS_ERR_UNSUPPORTED, "%.3g rows of queries in one call", (double)B * a.H * a.n);
    const int64_t rows = B * a.H * a.n;
    if (rows == 0) return FS_OK;
    a.lse = lse;
    a.ctx_len = t->ctx_len;
    a.parents = t->parents;
    a.parents_stride = t->parents_stride;
    a.q_vec = attn::aligned16(a.q, a.c.B, a.n, a.H);
    NvtxRange range("fs_tree_attention");
    Call c;
    int sms = 0;
    FS_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    const int per_head = a.R * a.n;
    const bool few = few_rows(a);
    TcArgs tc = {};
    int splits;
    if (few) {
        int resident = 0;
        p.row_blocks = per_head <= 8 || a.c.held == kv::HELD_16 ? 1 : 2;
        p.groups = (per_head + 8 * p.row_blocks - 1) / (8 * p.row_blocks);
        FS_CUDA(few_resident(a, p.row_blocks, &resident));
        splits = choose_few_splits(B * a.c.G * p.groups, a.c.reach(), (int64_t)sms * resident,
                                   a.c.held != kv::HELD_16);
    } else {
        tc.groups = (per_head + 255) / 256;
        tc.o_vec = attn::aligned16(a.o, a.c.B, a.n, a.H);
        splits = choose_tc_splits(B * a.c.G * tc.groups, a.c.reach(), sms);
    }
    Partials part = {};
    part.rows = rows;
    size_t part_out = 0, part_lse = 0;
    if (splits > 1) {
        part_out = c.L.take(sizeof(float) * (size_t)splits * rows * a.d);
        part_lse = c.L.take(sizeof(float) * (size_t)splits * rows);
    }
    const bool scratch = c.L.off > 0;
    FS_TRY(begin_call(c, stream, scratch));
    FS_TRY(ensure_capacity(c));
    if (scratch) {
        part.out = c.at<float>(part_out);
        part.lse2 = c.at<float>(part_lse);
    }
    a.err = c.ws->err_word;
    if (few) {
        p.part = part;
        p.splits = splits;
        p.counters = c.ws->counters;
        FS_CUDA(launch_few(p, c.stream));
    } else {
        tc.a = a;
        tc.part = part;
        tc.splits = splits;
        FS_TRY(tc_maps(tc, a.bf16));
        FS_CUDA(launch_tc(tc, c.stream));
        if (splits > 1) {
            attn::Args j = {};
            j.o = a.o;
            j.B = a.c.B;
            j.H = a.H;
            j.n = a.n;
            j.d = a.d;
            j.bf16 = a.bf16;
            j.lse = a.lse;
            FS_CUDA(attn::launch_combine(j, part, splits, c.stream));
        }
    }
    return scratch ? end_call(c) : FS_OK;
}

}  // namespace

}  // namespace tree
}  // namespace fs

using namespace fs;

extern "C" fs_status fs_tree_attention(const fs_cache* cache, const fs_tree* tree, const void* q, void* out,
                                       float* lse, void* stream) {
    try {
        return tree::tree_entry(cache, tree, q, out, lse, stream);
    } catch (...) {
        return fail(FS_ERR_CUDA, "unexpected host exception");
    }
}
