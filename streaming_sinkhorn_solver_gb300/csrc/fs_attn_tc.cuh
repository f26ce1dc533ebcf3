// Tensor-core building blocks of the cross-attention kernels, beyond those of
// fs_tc.cuh: tensor-map copies of 64 x 128 boxes of a (batch, token, head, d)
// tensor, tcgen05.mma with its A operand in TMEM, and operand tiles read with
// their rows as the summed dimension.
//
// Shared-memory tiles: 128 tokens x 64 elements, one 128-byte row per token in
// the 128-byte swizzle (tc::CHUNK_BYTES); a head of d > 64 takes two, one after
// the other.  Such a tile is an operand over d (K-major) for the score
// products, and over tokens (MN-major: the d elements are contiguous) for the
// products that sum over tokens.
#pragma once

#include "fs_attn.cuh"
#include "fs_tc.cuh"

#include <cuda.h>

namespace fs {
namespace attn {

using namespace fs::tc;

constexpr int kTile = 128;   // tokens of a tile

__device__ __forceinline__ uint64_t mul2f(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int c0, int token, int head,
                                         int batch, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(token), "r"(head), "r"(batch), "r"(smem_u32(bar))
        : "memory");
}

// A whole warp waits; its lanes agree on the result and are joined for the
// warp-collective instructions that follow.  (One lane waiting for the others and
// a broadcast took 4 to 12 % longer over the forward pass, 8 % over the gradients.)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* err, uint32_t code) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, err, code));
}
// The issuing thread's wait for a barrier, ordered before its products.
__device__ __forceinline__ bool mma_wait(uint32_t* err, uint64_t* bar, uint32_t phase) {
    const bool ok = mbar_wait(bar, phase, err, ERR_TIMEOUT_MMA);
    tc_fence_after();
    return ok;
}

// Whether the phase of parity `phase` has completed, without waiting.  A completed wait
// takes 100 to 160 cycles; tests sent ahead of other work or of one another hide that.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t phase) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(phase)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// one lane of a converged warp: the issuer of its copies and products
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]; A holds two 16-bit elements of a row per column
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                           uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Operand summed over the tokens of a tile: element (token, c) at row token of
// the 64-element chunk c / 64.  Groups of 8 tokens are 1024 bytes apart, the
// next 64 elements a chunk apart; 16 tokens on, the start address is 2048 bytes up.
__device__ __forceinline__ uint64_t sdesc_tokens(uint32_t saddr, uint32_t chunk_bytes = CHUNK_BYTES) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(chunk_bytes >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Operand of 16 elements a row without swizzle: 8 x 8 element blocks of 128 bytes
// (rows of 16 bytes), the two of a row group `second` bytes apart, row groups `group`.
__device__ __forceinline__ uint64_t sdesc_flat(uint32_t saddr, uint32_t second, uint32_t group) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(second >> 4) << 16;
    d |= (uint64_t)(group >> 4) << 32;
    d |= (uint64_t)1 << 46;
    return d;
}

// kind::f16 with float32 sums; b_tokens: B is summed over its rows
__host__ __device__ constexpr uint32_t idesc_16(bool bf16, int N, bool b_tokens) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) |
           ((b_tokens ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// 32 lanes x 16 columns: thread t gets lane t
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]),
          "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}

// D[tmem] = A * B^T over the d elements of a 128-token tile (A) and a tile of
// B_CHUNK / 128 tokens (B), in chunks of 64, both zero beyond d; `turns` times U products
// of 16 elements.  The issuing thread takes 80 cycles for a product a turn, 45 with two,
// 32 with four: with U = 4 the forward pass of heads of 128 takes 120 us for 128 (U = 1)
// and 124 (U = 2), of heads of 80 114 for 120, although it adds zeros there.  U = 2 where
// a product takes longer than that anyway.
//
// Every product is issued by the one lane that elect.sync names, in code inlined into that
// lane's branch, and the sizes of a product's operands are constants of the code; run-time
// counts are loop bounds, and conditions stand around whole groups of products and their
// commit.  (A first version issued them from a function that was not inlined, under
// `lane == 0`, with a condition around each product, and ended in illegal accesses with
// the operands that are right here.  All three went at once; which of them it was is not known.)
template <int U, int B_CHUNK = CHUNK_BYTES>
__device__ __forceinline__ void mma_over_d(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                           int turns) {
#pragma unroll 1
    for (int x = 0; x < turns; ++x) {
        const int chunk = x * U / 4, step = x * U % 4;
        const uint64_t da = a + (uint64_t)(chunk * (CHUNK_BYTES >> 4) + 2 * step);
        const uint64_t db = b + (uint64_t)(chunk * (B_CHUNK >> 4) + 2 * step);
#pragma unroll
        for (int y = 0; y < U; ++y) mma_f16(d_tmem, da + 2 * y, db + 2 * y, idesc, x != 0 || y != 0);
    }
}
// the same with A in TMEM, a chunk of 64 a turn
__device__ __forceinline__ void mma_over_d_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                              int chunks) {
#pragma unroll 1
    for (int x = 0; x < chunks; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y)
            mma_f16_ts(d_tmem, a_tmem + 32 * x + 8 * y, b + (uint64_t)(x * (CHUNK_BYTES >> 4) + 2 * y), idesc,
                       x != 0 || y != 0);
}
// D[tmem] (+)= A[tmem] * B over the KEYS tokens of B's tile; tokens 64 and on of A are
// `half` columns from its first.  One elected thread.
template <int KEYS = kTile>
__device__ __forceinline__ void mma_over_tokens(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                                uint32_t idesc, bool accumulate, uint32_t half) {
#pragma unroll
    for (int x = 0; x < KEYS / 16; ++x)
        mma_f16_ts(d_tmem, a_tmem + (x >> 2) * half + 8 * (x & 3), b + 128 * x, idesc,
                   accumulate || x != 0);
}

// Forward, p = 2^{x - ref + kProbShift}: up to 2^8 without the shift, whose largest value
// float16 would use half of its range for.  With it float16 holds p in full from 2^-21 of
// the reference's weight on and rounds to multiples of 2^-31 of it below (without it from
// 2^-14, and weights below 2^-25 were in the sum of p but not in out: all that 200000 keys 18
// below one other bring).  The type's end, 65504, is above 2^15.  bfloat16 has float32's range.
template <bool BF>
constexpr float kProbShift = BF ? 0.f : 7.f;

// two floats rounded to one register, x in the low half
template <bool BF>
__device__ __forceinline__ uint32_t pack16(float x, float y) {
    uint32_t r;
    if (BF)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    return r;
}

// One row of the 32 of a warp, 16 elements [c, c + 16) in o, rounded into a tile of
// 128 rows x 64 elements (chunks on chunks) in the 128-byte swizzle.
template <bool BF>
__device__ __forceinline__ void stage16(uint8_t* tile, int r, int c, const float* o) {
#pragma unroll
    for (int e = 0; e < 16; e += 8)
        *reinterpret_cast<uint4*>(tile + (c >> 6) * CHUNK_BYTES + swz_offset(r, (c & 63) + e)) =
            make_uint4(pack16<BF>(o[e], o[e + 1]), pack16<BF>(o[e + 2], o[e + 3]),
                       pack16<BF>(o[e + 4], o[e + 5]), pack16<BF>(o[e + 6], o[e + 7]));
}
// ROWS staged rows from r0 on, of which `rows` exist, to memory by a warp: eight lanes to
// 64 elements where the rows take 16-byte stores, else an element per lane.
template <int ROWS>
__device__ __forceinline__ void unstage_rows(const uint8_t* tile, int r0, int rows, int d, uint16_t* out,
                                             int64_t stride, bool vec, int lane) {
    __syncwarp();
    if (vec) {
        for (int c = 0; c < d; c += 64) {
            const int e = c + (lane & 7) * 8;
#pragma unroll
            for (int k = 0; k < ROWS; k += 4) {
                const int r = k + (lane >> 3);
                if (r < rows && e < d)
                    *reinterpret_cast<uint4*>(out + r * stride + e) = *reinterpret_cast<const uint4*>(
                        tile + (c >> 6) * CHUNK_BYTES + swz_offset(r0 + r, e & 63));
            }
        }
    } else {
        for (int r = 0; r < rows && r < ROWS; ++r)
            for (int e = lane; e < d; e += 32)
                out[r * stride + e] = *reinterpret_cast<const uint16_t*>(
                    tile + (e >> 6) * CHUNK_BYTES + swz_offset(r0 + r, e & 63));
    }
}

// Position in a ring of `n` stages: slot, and the parity its next use completes with.
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step(int by, int n) {
        slot += by;
        if (slot >= n) {
            slot -= n;
            phase ^= 1u;
        }
    }
};

// warp: 32 registers into 32 consecutive columns of the warp's lanes
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
        "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
        "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                     taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Tiles of 128 keys a sequence visits, and which of a tile's keys count.
struct KeyTiles {
    const uint4* words;     // [B][tiles] bits of counted keys, or nullptr (no mask)
    const int* list;        // [B][tiles] tiles with a counted key, in order
    const int* count;       // [B]
    int tiles;              // ceil(m / 128)
};
// counted keys of a tile as 128 bits
__device__ __forceinline__ uint4 tile_words(const KeyTiles& kt, int b, int tile, int end) {
    if (kt.words) return __ldg(kt.words + (int64_t)b * kt.tiles + tile);
    const int left = end - tile * kTile;   // >= 1
    auto w = [&](int k) -> uint32_t {
        const int c = left - 32 * k;
        return c <= 0 ? 0u : (c >= 32 ? 0xffffffffu : (1u << c) - 1u);
    };
    return make_uint4(w(0), w(1), w(2), w(3));
}

// The same in steps of KT = 128 or 64 keys: their count, first key, and bits.
template <int KT>
__device__ __forceinline__ int step_count(const KeyTiles& kt, int b, int end) {
    return kt.list ? __ldg(kt.count + b) * (kTile / KT) : (end + KT - 1) / KT;
}
template <int KT>
__device__ __forceinline__ int step_key(const KeyTiles& kt, int b, int j) {
    if (!kt.list) return j * KT;
    constexpr int per = kTile / KT;
    return __ldg(kt.list + (int64_t)b * kt.tiles + j / per) * kTile + (j % per) * KT;
}
// The sequence that the blocks of rank b take, by whole warps: those with more keys first,
// so that the last turn of the GPU's blocks is of short ones (8 x 500 queries of 600 to
// 1500 keys, 16 heads of 64: 40 us for 42.5).  Under a mask (the counts are a load further
// away: 68 us for 64 there) and beyond 32 sequences in their own order.
template <int KT>
__device__ __forceinline__ int longest_first(const KeyTiles& kt, const Args& a, int b) {
    if (a.B == 1 || a.B > 32 || kt.list || !a.kv_len) return b;
    const int lane = threadIdx.x & 31;
    const int steps = lane < a.B ? step_count<KT>(kt, lane, key_end(a, lane)) : -1;
    int rank = 0;
    for (int k = 0; k < a.B; ++k) {
        const int other = __shfl_sync(0xffffffffu, steps, k);
        rank += other > steps || (other == steps && k < lane);
    }
    return __ffs(__ballot_sync(0xffffffffu, lane < a.B && rank == b)) - 1;
}

template <int KT>
struct KeyBits {
    uint32_t w[KT / 32];
    __device__ __forceinline__ KeyBits(const KeyTiles& kt, int b, int j, int end) {
        const int key = step_key<KT>(kt, b, j);
        const uint4 all = tile_words(kt, b, key / kTile, end);
        if (KT == kTile) {
            w[0] = all.x;
            w[1] = all.y;
            w[KT / 32 - 2] = all.z;
            w[KT / 32 - 1] = all.w;
        } else {
            w[0] = key & 64 ? all.z : all.x;
            w[1] = key & 64 ? all.w : all.y;
        }
    }
    __device__ __forceinline__ bool all() const {
        uint32_t x = w[0];
#pragma unroll
        for (int k = 1; k < KT / 32; ++k) x &= w[k];
        return x == 0xffffffffu;
    }
};

// One whole warp: zeroes the rows of a landed tile whose keys do not count (what
// such keys hold would otherwise enter sums as 0 * NaN).
template <int KT>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int chunks, int chunk_bytes, const KeyBits<KT>& w,
                                           int lane) {
    // 8 lanes clear a 128-byte row, stores under a predicate (branches take four times as long)
    const uint32_t at = smem_u32(tile) + (lane >> 3) * 128 + (lane & 7) * 16;
#pragma unroll
    for (int k = 0; k < KT / 32; ++k) {
        if (w.w[k] == 0xffffffffu) continue;
        const uint32_t bits = w.w[k] >> (lane >> 3);
        for (int c = 0; c < chunks; ++c) {
#pragma unroll
            for (int r4 = 0; r4 < 32; r4 += 4)
                asm volatile(
                    "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %0, 0;\n\t"
                    "@p st.shared.v4.u32 [%1], {%2, %2, %2, %2};\n\t}" ::"r"((bits >> r4) & 1u),
                    "r"(at + c * chunk_bytes + (32 * k + r4) * 128), "r"(0)
                    : "memory");
        }
    }
}

// A tile's mask as an operand: a product with it adds -inf to the scores of the keys
// that do not count, so the softmax has no test per score (batch 4, 2048 x 2048, 16 heads
// with 3 % of the keys masked: 100 us for 125 with heads of 64, 135 for 157 with 128).  Rows of 16 elements, bfloat16 whatever
// the type: 0 or -inf, then zeros; the second half of every row is one block of zeros
// that all tiles share.  The other operand has ones in the first column.
template <int KT, int TILES>
struct KeyMask {
    static constexpr int kTileBytes = KT * 16, kOnes = TILES * kTileBytes, kZeros = kOnes + kTile * 16;
    static constexpr int kBytes = kZeros + kTile * 16;
    uint8_t* p;
    // every thread of the block, before it meets
    __device__ __forceinline__ void init(int t, int threads) const {
        for (int e = t; e < 2 * kTile; e += threads)
            reinterpret_cast<uint4*>(p + kOnes)[e] = make_uint4(e < kTile ? 0x3f80u : 0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    // One whole warp, before the fence and the arrival that publish the tile
    __device__ __forceinline__ void write(int slot, const KeyBits<KT>& w, int lane) const {
#pragma unroll
        for (int k = 0; k < KT / 32; ++k)
            reinterpret_cast<uint4*>(p + slot * kTileBytes)[32 * k + lane] =
                make_uint4((w.w[k] >> lane) & 1u ? 0u : 0xff80u, 0u, 0u, 0u);
    }
    // descriptors of the ones and of a tile's mask, kStep more from a tile to the next
    static constexpr uint64_t kStep = (uint64_t)(kTileBytes >> 4) - ((uint64_t)(kTileBytes >> 4) << 16);
    __device__ __forceinline__ uint64_t ones() const {
        return sdesc_flat(smem_u32(p) + kOnes, kZeros - kOnes, 128);
    }
    __device__ __forceinline__ uint64_t tile(int slot) const {
        return sdesc_flat(smem_u32(p), kZeros, 128) + slot * kStep;
    }
};

}  // namespace attn
}  // namespace fs
