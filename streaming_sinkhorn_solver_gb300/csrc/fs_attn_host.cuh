// Launch interfaces of the cross-attention kernels.
#pragma once

#include "fs_attn_tc.cuh"
#include "fs_host.cuh"

#include <algorithm>
#include <atomic>

namespace fs {
namespace attn {

// keys of a tile of the forward kernel
constexpr int forward_keys(int d) { return d <= 64 ? 128 : 64; }

// A tensor as 64 x 128 boxes of (d, token, head, batch); a repeated (stride 0)
// head or batch is one entry of the map, its index multiplied by 0.
struct TensorMap {
    CUtensorMap map;
    int head, batch;   // index factors, 0 or 1
};

// Row sums over part of the keys, joined by k_combine: rows are (b, h, i)
struct Partials {
    float* out;        // [splits][rows][d], divided by its own sum
    float* lse2;       // [splits][rows], base 2
    int64_t rows;
};

struct FwdArgs {
    TensorMap q, k, v;
    Args a;
    KeyTiles kt;
    Partials part;
    int row_blocks, splits;
    int out_vec;       // the rows of out take 16-byte stores
};

// -lse2 / scale2 and -delta of 128 queries, each as three bfloat16 terms, in the form
// of an operand of 16 elements a row (sdesc_flat), kRowBytes; then -lse2 and -delta in
// float32
constexpr int kRowBytes = kTile * 32, kRowStride = kRowBytes + 8 * kTile;

struct GradArgs {
    TensorMap q, k, v, dout;
    Args a;
    KeyTiles kt;
    uint8_t* rows;     // [B][H][q_tiles][kRowStride]: row values of the queries
    int q_tiles, k_tiles;
    bool exact_delta;  // from the scores (k_grad_delta), not from O
    // where few blocks have many tiles: shares of a block's tiles, and their sums in float32
    // (rows (b, head, token); delta: rows of rows), joined in order
    int q_splits, k_splits;
    float *part_dq, *part_dk, *part_dv, *part_delta;
    // float16: what bounds |ds| (range_shift).  For every 32 queries, [B][H][q_tiles][4]: a
    // bound on theirs with exact_delta, else the largest norm of their dO; that goes with
    // the largest norm of a counted value of each key tile, [B][G][k_tiles]
    float *q_range, *v_range, *part_top;
    int stages, kv_stages, delta_stages, scratch_rows;     // set at launch
    int dout_vec, o_vec, dq_vec, dk_vec, dv_vec;   // rows take 16-byte accesses
};

// dq, then dk and dv, then dbias (nullptr: none)
cudaError_t launch_grad_tc(const GradArgs& p, void* dbias, cudaStream_t s);
cudaError_t launch_forward_tc(const FwdArgs& p, cudaStream_t s);

// Few query rows per key head: row_blocks of 8 rows to a block (1 or 2), in `groups`.
struct DecodeArgs {
    Args a;
    Partials part;
    int splits, groups, row_blocks;
    int dp;                // elements of a partial row: d, to a multiple of 4
    unsigned* counters;    // [batch x key heads x groups], zero between calls
};
constexpr int kDecodeKeys = 128;           // the splits are whole multiples of these keys
cudaError_t launch_decode(const DecodeArgs& p, cudaStream_t s);
// blocks of it that an SM holds
cudaError_t decode_resident(const Args& a, int row_blocks, int* blocks);
cudaError_t launch_combine(const Args& a, const Partials& part, int splits, cudaStream_t s);
cudaError_t launch_key_tiles(const Args& a, uint4* words, int* list, int* count, int tiles,
                             cudaStream_t s);
// out = 0, lse = -inf (no keys), or zero gradients
cudaError_t launch_zero(const Args& a, const View& w, int tokens, int heads, float* lse, cudaStream_t s);
// contiguous copy of a (batch, token, head, d) tensor with rows of dp elements, zero beyond d
cudaError_t launch_pack(const View& from, void* to, int B, int tokens, int heads, int d, int dp,
                        cudaStream_t s);

// Raises a kernel's limit of dynamic shared memory, once per device.
template <typename K>
cudaError_t raise_smem(K kernel, size_t bytes, std::atomic<uint64_t>& ready) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!(ready.load() >> dev & 1)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != cudaSuccess) return e;
        ready.fetch_or(1ull << dev);
    }
    return cudaSuccess;
}

// boxes of `rows` tokens
fs_status make_tensor_map(TensorMap& t, const View& w, int B, int tokens, int heads, int d, bool bf16,
                          int rows = kTile);
}  // namespace attn
}  // namespace fs
