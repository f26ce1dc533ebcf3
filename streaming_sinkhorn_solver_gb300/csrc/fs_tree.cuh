// Launch interfaces of the tree attention's kernels.
//
// Rows of a sequence and key head are (token t, query head r of the R that share it),
// row = t R + r.  Keys are positions: below `ctx` all rows see them, from there on they are
// the tree's tokens, and bits say which of them a token sees.
#pragma once

#include "fs_kv.cuh"

namespace fs {
namespace tree {

using attn::Partials;
using attn::View;
using kv::Cache;

struct Args {
    Cache c;
    View q, o;
    int H, R, n, d;
    int bf16;
    int q_vec;                   // the rows of q take 16-byte loads
    float scale2;                // scale log2(e)
    float* lse;                  // [B][H][n], natural logarithm
    const int32_t* ctx_len;      // [B]
    const int32_t* parents;      // rows of n, or nullptr (a chain)
    int64_t parents_stride;
    uint32_t* err;               // device error word
};

__device__ __forceinline__ int context(const Args& a, int b) {
    const int l = __ldg(a.ctx_len + b);
    return l < 0 ? 0 : min(l, a.c.reach());
}

// 2^n, -126 <= n <= 127
__device__ __forceinline__ float two_to(int n) { return __int_as_float((127 + n) << 23); }

// Queries in bfloat16 beside an 8-bit cache become float16, each row times the power of two that
// brings its largest finite magnitude to [2^14, 2^15): float16 holds elements from 2^-31 of that on to all
// their bits, others to 2^-39 of it.  (One power for a block of any rows left nothing of a row
// beside one 2^40 times as large.)
// top: the larger of it and two bfloat16 magnitudes
__device__ __forceinline__ uint32_t finite_top(uint32_t top, uint32_t w) {
    const uint32_t l = w & 0x7fffu, h = w >> 16 & 0x7fffu;
    return max(top, max(l < 0x7f80u ? l : 0u, h < 0x7f80u ? h : 0u));
}
__device__ __forceinline__ int query_shift(uint32_t top) { return min(14 + 127 - (int)(top >> 7), 126); }
__device__ __forceinline__ uint32_t shifted_pair(uint32_t w, float up) {
    return attn::pack16<false>(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
}

// What a token of the tree sees of it: bit u for token u, none if it is not there.
constexpr int kTreeWords = kv::kMaxTree / 32;
// parents: in shared memory, or nullptr for a chain
__device__ __forceinline__ void tree_row(const int* parents, int t, uint32_t* words) {
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w) words[w] = 0;
    if (parents == nullptr) {
        for (int w = 0; w <= t >> 5; ++w) words[w] = w < t >> 5 ? 0xffffffffu : (2u << (t & 31)) - 1u;
        return;
    }
    int u = t;
    while (u >= 0) {
        words[u >> 5] |= 1u << (u & 31);
        const int up = parents[u];
        if (up >= u || up < -1) {         // no parent: the token is not there
#pragma unroll
            for (int w = 0; w < kTreeWords; ++w) words[w] = 0;
            return;
        }
        u = up;
    }
}
// 32 keys from key `at` of the tree on (above -32), as a row sees them; the keys before
// the tree too, where the row is there.
__device__ __forceinline__ uint32_t tree_window(const uint32_t* words, bool there, int at) {
    if (!there) return 0;
    if (at < 0) return at <= -32 ? 0xffffffffu : words[0] << -at | ((1u << -at) - 1u);
    if (at >= kv::kMaxTree) return 0;
    const int w = at >> 5;
    return __funnelshift_r(words[w], w + 1 < kTreeWords ? words[w + 1] : 0u, at & 31);
}

// Few rows: row_blocks of 8 rows to a block (1; in 8 bits or 2), in `groups`.
struct FewArgs {
    Args a;
    Partials part;
    int splits, groups, row_blocks;
    unsigned* counters;    // [batch x key heads x groups], zero between calls
};
constexpr int kFewKeys = 128;          // the splits are whole multiples of these keys
cudaError_t launch_few(const FewArgs& p, cudaStream_t s);
// blocks of it that an SM holds
cudaError_t few_resident(const Args& a, int row_blocks, int* blocks);

// Many rows, on the tensor cores: `groups` of 256 rows, or one of up to 128.
struct TcArgs {
    CUtensorMap k, v;      // (d, token, head, page)
    Args a;
    Partials part;         // rows of d floats
    int splits, groups;
    int o_vec;             // the rows of out take 16-byte stores
};
constexpr int kTcKeys = 64;            // keys of a tile
// whether the cache's copies can be described to it
bool tc_copies(const Cache& c);
fs_status tc_maps(TcArgs& p, bool bf16);
cudaError_t launch_tc(const TcArgs& p, cudaStream_t s);

}  // namespace tree
}  // namespace fs
