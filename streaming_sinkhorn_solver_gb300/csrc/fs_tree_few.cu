// Tree attention, few query rows per key head: bound by reading the cache once.
//
// As in the cross attention of few queries, the rows that share a key head are one tile of
// 8 (or 16, of 8-bit caches that have no copies by the page), blocks split the keys, and a warp takes 32 keys at a time straight from memory
// into the operand registers of mma.sync (S = Q K^T with any 16 of the d elements in a
// product, the same for both operands; O^T += V^T P^T, with P^T in S's own layout).
//
// A cache in 8 bits comes through a ring in shared memory that each warp keeps for itself,
// two steps ahead by asynchronous copies, and is widened to float16 in registers, which is
// exact: a lane's 16 bytes of a key row are 4 products' worth of its operand, and of four value
// rows a byte permute pairs two keys before they are widened.  (Straight from memory, as the 16-bit
// types come, the loads of a step waited for the page numbers and the products for the loads,
// with registers for two blocks to an SM: half the speed.)  Scales stay in float32:
//   w_ij = q_i . code_j (scale2 ks_j),   x_ij = w_ij + log2 vs_j,   P_ij = 2^{x_ij - ref_i},
//   O_i = sum_j P_ij code_j,   sum_i = sum_j 2^{w_ij - ref_i},
// so that the largest P of a row is the one that counts most in O, whatever the scales,
// and float16 holds them all as it holds weights.  The sum's terms are up to 2^8 / vs_j, 2^97 for the
// least scale that a row can have, and the one of the reference is 1 / vs, 2^-122 or more: float32
// holds them all.  (The sum as that of P_ij / vs_j has the same price, a reciprocal for an
// exponential, but takes 0 / vs_j from keys that a row does not see.)  Queries in bfloat16 become
// float16, each row times a power of two (query_shift).
//
// Measured, 8 key heads of 128, 4 rows: 38 sequences of 8192 e4m3 keys 117 to 120 us, 5.5 TB/s (0.81
// of the measured copy rate; DRAM at 69 % of its peak, issue slots at 47 %: the latency of a warp's
// steps, with 8 warps to an SM); one sequence of 2000 bfloat16 keys 10 us, latency.
#include "fs_tree.cuh"

#include <type_traits>

namespace fs {
namespace tree {

namespace {

using namespace fs::attn;
using kv::HELD_16;
using kv::HELD_E4M3;
using kv::HELD_I8;

constexpr int kWarps = 4;
constexpr int kWords = kTreeWords + 1;     // (odd: rows in banks of their own)

template <bool BF>
__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ld16(const uint8_t* p, bool on, uint32_t* x) {
    x[0] = x[1] = x[2] = x[3] = 0;
    if (on)
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                     : "l"(p));
}

// whether a register of the held type has an element that is not finite
template <int HELD, bool BF>
__device__ __forceinline__ bool nonfinite(uint32_t w) {
    if (HELD == HELD_I8) return false;
    if (HELD == HELD_E4M3) {
        const uint32_t m = w & 0x7f7f7f7fu;       // a byte of 0x7f
        return ((m + 0x01010101u) & 0x80808080u) != 0;
    }
    constexpr uint32_t kExp = BF ? 0x7f80u : 0x7c00u;
    return (w & kExp) == kExp || ((w >> 16) & kExp) == kExp;
}

__device__ __forceinline__ void cp16(uint32_t dst, const uint8_t* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const uint8_t* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(on ? 8 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const float* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0)
                 : "memory");
}

// 8 bits, a warp's step of 32 keys in shared memory: codes of keys, of values, scales of both.
// Rows of 128 bytes (two rows of 64 elements to one); the 16-byte unit u of row r lies where
// the lanes that read at once (keys: two rows, half of each; values: two units of rows 2 t)
// find theirs in different banks.
template <int HD>
struct Step {
    static constexpr int kSteps = 3;
    static constexpr int kRows = 32 * HD, kScales = 2 * 32 * 4;
    static constexpr int kBytes = 2 * kRows + kScales;
    __device__ static __forceinline__ int key_at(int r, int u) {
        return HD == 128 ? 128 * r + 16 * (u ^ ((r & 1) << 2)) : value_at(r, u);
    }
    __device__ static __forceinline__ int value_at(int r, int u) {
        return HD == 128 ? 128 * r + 16 * (u ^ (2 * (r >> 1 & 3)))
                         : 128 * (r >> 1) + 16 * (((r & 1) * 4 + u) ^ (2 * (r >> 1 & 3)));
    }
};

// RB: blocks of 8 query rows.  A warp's rows of O lie over its ring.
template <int HD, int HELD, int RB>
constexpr int kWarpBytes = HELD == HELD_16 || Step<HD>::kSteps * Step<HD>::kBytes < 4 * 8 * RB * HD
                               ? 4 * 8 * RB * HD
                               : Step<HD>::kSteps * Step<HD>::kBytes;
template <int HD, int HELD, int RB>
constexpr size_t kFewSmem = kWarps * (kWarpBytes<HD, HELD, RB> + sizeof(float) * 2 * 8 * RB);

template <int HD, int HELD, bool BF, int RB>
__global__ void __launch_bounds__(32 * kWarps) k_tree_few(const __grid_constant__ FewArgs P) {
    using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    constexpr bool Q8 = HELD != HELD_16;
    constexpr bool MB = BF && !Q8;                    // products in bfloat16
    constexpr int EB = Q8 ? 1 : 2;                    // bytes of an element
    constexpr int PIECE = 16 / EB;                    // elements of a key piece
    constexpr int U = HD / (4 * PIECE);               // key pieces of a lane
    constexpr int VW = HD * EB / 32;                  // registers of a lane's part of a value row
    constexpr int NT = HD / 16;                       // O tiles: two elements of d to a lane
    constexpr int KB = !Q8 && HD == 64 ? 1 : 2, KEYS = 16 * KB;
    constexpr int kWarpRows = kWarpBytes<HD, HELD, RB> / 4;     // floats from a warp's rows to the next's
    constexpr int RP = (RB + 1) / 2, ROWS = 8 * RB;
    constexpr float kShift = kProbShift<MB>;
    extern __shared__ float smem[];
    float* sO = smem;                                   // [warp][row][HD]
    float* sRef = sO + kWarps * kWarpRows;              // [warp][row]
    float* sSum = sRef + kWarps * ROWS;
    __shared__ int sParents[kv::kMaxTree];
    __shared__ uint32_t sTree[ROWS][kWords];
    __shared__ int sLast;
    const Args& a = P.a;
    const Cache& c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;

    int blk = blockIdx.x;
    const int split = blk % P.splits;
    blk /= P.splits;
    const int group = blk % P.groups;
    blk /= P.groups;
    const int kh = blk % c.G;
    const int b = blk / c.G;
    const int nrows = min(ROWS, a.R * a.n - group * ROWS);
    const int ctx = context(a, b);
    const int end = min(ctx + a.n, c.reach());
    // this split's keys, in whole steps of the block
    const int steps = (end + kFewKeys - 1) / kFewKeys;
    const int per = (steps + P.splits - 1) / P.splits;
    const int k0 = (int)min((int64_t)end, (int64_t)split * per * kFewKeys);
    const int k1 = (int)min((int64_t)end, k0 + (int64_t)per * kFewKeys);

    // what each row sees of the tree
    if (a.parents) {
        const int32_t* p = a.parents + b * a.parents_stride;
        for (int e = threadIdx.x; e < a.n; e += 32 * kWarps) sParents[e] = __ldg(p + e);
        __syncthreads();
    }
    if (threadIdx.x < ROWS) {
        const int row = group * ROWS + min((int)threadIdx.x, nrows - 1);
        tree_row(a.parents ? sParents : nullptr, row / a.R, sTree[threadIdx.x]);
    }

    // Row 8 rb + g of the tile: its queries as the products' operand
    uint32_t q[RB][U][4 * (Q8 ? 2 : 1)];
    float mul[RB];                        // scale2, over what the row was multiplied by
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int row = group * ROWS + min(8 * rb + g, nrows - 1);
        const int tok = row / a.R, r = row - tok * a.R;
        const uint16_t* p = static_cast<const uint16_t*>(a.q.p) + b * a.q.sb + tok * a.q.st +
                            (int64_t)(kh * a.R + r) * a.q.sh;
        mul[rb] = a.scale2;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int x = 0; x < (Q8 ? 2 : 1); ++x) {
                const int e = PIECE * (t + 4 * u) + 8 * x;
                uint32_t* w = q[rb][u] + 4 * x;
                if (a.q_vec) {
                    ld16(reinterpret_cast<const uint8_t*>(p + e), e < a.d, w);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = e < a.d ? (uint32_t)p[e + 2 * k] | (uint32_t)p[e + 2 * k + 1] << 16 : 0u;
                }
            }
        if (Q8 && BF) {
            uint32_t top = 0;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < 8; ++k) top = finite_top(top, q[rb][u][k]);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int up = query_shift(top);
            mul[rb] = a.scale2 * two_to(-up);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < 8; ++k) q[rb][u][k] = shifted_pair(q[rb][u][k], two_to(up));
        }
    }
    __syncthreads();
    bool there[RB];
    const uint32_t* words[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int row = group * ROWS + min(8 * rb + g, nrows - 1), tok = row / a.R;
        words[rb] = sTree[min(8 * rb + g, nrows - 1)];
        there[rb] = words[rb][tok >> 5] >> (tok & 31) & 1u;
    }
    float ref[RB], sum[RB], o[RB][NT][4];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        ref[rb] = -INFINITY;
        sum[rb] = 0.f;
#pragma unroll
        for (int w = 0; w < NT; ++w)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[rb][w][e] = 0.f;
    }
    const uint8_t* kp = c.k.p + kh * c.k.head;
    const uint8_t* vp = c.v.p + kh * c.v.head;

    // 8 bits: the ring, and what of the steps in it counts
    using St = Step<HD>;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * 4 * kWarpRows;
    uint32_t next_bits[St::kSteps - 1];
#pragma unroll
    for (int x = 0; x < St::kSteps - 1; ++x) next_bits[x] = 0;
    int entry = -1;                       // of the step to be asked for, its keys 8 (lane & 3) on
    const auto load_entry = [&](int key) {
        const int i = (key + 8 * (lane & 3)) >> c.log_page;
        int e = -1;
        if (key < k1 && i < c.table_pages)
            asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(e) : "l"(c.table + b * c.table_stride + i));
        return e;
    };
    constexpr int kUnits = HD / 16, kStep = 32 / kUnits;      // of a row; rows of an access
    const int unit = lane % kUnits;
    const bool whole = c.vec16 && a.d == HD;
    const int64_t k_off = (lane / kUnits) * c.k.token + 16 * unit, k_far = kStep * c.k.token;
    const int64_t v_off = (lane / kUnits) * c.v.token + 16 * unit, v_far = kStep * c.v.token;
    const float* k_scale = c.k.scale + kh * c.k.s_head;
    const float* v_scale = c.v.scale + kh * c.v.s_head;
    const auto ask = [&](int key, int stage) -> uint32_t {
        const uint32_t to = ring + stage * St::kBytes;
        const int left = k1 - (key + 8 * (lane & 3));
        const bool on = (unsigned)entry < c.pages && left > 0;
        const int held = on ? entry : -1;
        entry = load_entry(key + KEYS * kWarps);
        uint32_t bits = on && lane < 4 ? (left >= 8 ? 255u : (1u << left) - 1u) << (8 * lane) : 0u;
        bits = __reduce_or_sync(0xffffffffu, bits);
        if (bits == 0xffffffffu && whole) {
            // All of them, in whole pieces: where each 8 begin comes from the lane that has their page.
            // (The general case below takes 25 instructions a copy; the kernel was bound by them.)
            const int slot0 = c.slot_of(key + 8 * (lane & 3));
            const uint8_t* kb = kp + held * c.k.page + slot0 * c.k.token;
            const uint8_t* vb = vp + held * c.v.page + slot0 * c.v.token;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint8_t* ks = reinterpret_cast<const uint8_t*>(
                                        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(kb), x)) + k_off;
                const uint8_t* vs = reinterpret_cast<const uint8_t*>(
                                        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(vb), x)) + v_off;
#pragma unroll
                for (int y = 0; y < 8 / kStep; ++y) {
                    const int r = 8 * x + y * kStep + lane / kUnits;
                    cp16(to + St::key_at(r, unit), ks + (y ? k_far : 0), true);
                    cp16(to + St::kRows + St::value_at(r, unit), vs + (y ? v_far : 0), true);
                }
            }
            const int pg = __shfl_sync(0xffffffffu, held, lane >> 3), slot = c.slot_of(key + lane);
            cp4(to + 2 * St::kRows + 4 * lane, k_scale + pg * c.k.s_page + slot, true);
            cp4(to + 2 * St::kRows + 4 * (32 + lane), v_scale + pg * c.v.s_page + slot, true);
            return bits;
        }
        const int u = unit;
#pragma unroll 1
        for (int i = 0; i < 32 / kStep; ++i) {
            const int pg = __shfl_sync(0xffffffffu, held, i * kStep / 8), r = i * kStep + lane / kUnits;
            const bool there = bits >> r & 1u;
            const int slot = c.slot_of(key + r);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const kv::Pool& p = v ? c.v : c.k;
                const uint8_t* src = there ? (v ? vp : kp) + pg * p.page + slot * p.token + 16 * u : p.p;
                const uint32_t dst = to + v * St::kRows + (v ? St::value_at(r, u) : St::key_at(r, u));
                if (c.vec16) {
                    cp16(dst, src, there && 16 * u < a.d);
                } else {
                    const bool first = there && 16 * u < a.d, second = there && 16 * u + 8 < a.d;
                    cp8(dst, first ? src : p.p, first);
                    cp8(dst + 8, second ? src + 8 : p.p, second);
                }
            }
        }
        const int pg = __shfl_sync(0xffffffffu, held, lane >> 3);
        const bool there = bits >> lane & 1u;
        const int slot = c.slot_of(key + lane);
        cp4(to + 2 * St::kRows + 4 * lane, there ? c.k.scale + pg * c.k.s_page + kh * c.k.s_head + slot : c.k.scale,
            there);
        cp4(to + 2 * St::kRows + 4 * (32 + lane),
            there ? c.v.scale + pg * c.v.s_page + kh * c.v.s_head + slot : c.v.scale, there);
        return bits;
    };
    int stage = 0;
    if (Q8) {
        entry = load_entry(k0 + KEYS * warp);
#pragma unroll
        for (int x = 0; x < St::kSteps - 1; ++x) {
            const int key = k0 + KEYS * (warp + kWarps * x);
            if (key < k1) next_bits[x] = ask(key, x);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }

    for (int key = k0 + KEYS * warp; key < k1; key += KEYS * kWarps) {
        uint32_t bits = 0;
        uint32_t k[2 * KB][U][4], v[KB][4][VW];
        float ks[4 * KB], lv[4 * KB];                  // of keys 8 nb + 2 t + {0, 1}
        const uint8_t* step = reinterpret_cast<const uint8_t*>(smem) + warp * 4 * kWarpRows + stage * St::kBytes;
        if (Q8) {
            __syncwarp();                 // the step before is done with
            const int far = key + KEYS * kWarps * (St::kSteps - 1);
            const int to = stage == 0 ? St::kSteps - 1 : stage - 1;
            bits = next_bits[0];
#pragma unroll
            for (int x = 0; x + 1 < St::kSteps - 1; ++x) next_bits[x] = next_bits[x + 1];
            next_bits[St::kSteps - 2] = far < k1 ? ask(far, to) : 0u;
            asm volatile("cp.async.commit_group;" ::: "memory");
            asm volatile("cp.async.wait_group %0;" ::"n"(St::kSteps - 1) : "memory");
            __syncwarp();
            stage = stage == St::kSteps - 1 ? 0 : stage + 1;
            if (bits == 0) continue;
#pragma unroll
            for (int nb = 0; nb < 2 * KB; ++nb)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint4 x = *reinterpret_cast<const uint4*>(step + St::key_at(8 * nb + g, t + 4 * u));
                    k[nb][u][0] = x.x, k[nb][u][1] = x.y, k[nb][u][2] = x.z, k[nb][u][3] = x.w;
                }
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int j = 16 * kb + 2 * t + (x & 1) + 8 * (x >> 1);
                    const uint8_t* row = step + St::kRows;
                    if (HD == 128) {
                        const uint4 y = *reinterpret_cast<const uint4*>(row + St::value_at(j, g));
                        v[kb][x][0] = y.x, v[kb][x][1] = y.y;
                        v[kb][x][VW > 2 ? 2 : 0] = VW > 2 ? y.z : y.x;
                        v[kb][x][VW > 2 ? 3 : 1] = VW > 2 ? y.w : y.y;
                    } else {
                        const uint2 y = *reinterpret_cast<const uint2*>(row + St::value_at(j, g >> 1) + 8 * (g & 1));
                        v[kb][x][0] = y.x, v[kb][x][1] = y.y;
                    }
                }
#pragma unroll
            for (int nb = 0; nb < 2 * KB; ++nb) {
                const float* s = reinterpret_cast<const float*>(step + 2 * St::kRows) + 8 * nb + 2 * t;
                const float2 x = *reinterpret_cast<const float2*>(s), y = *reinterpret_cast<const float2*>(s + 32);
                kv::weigh(x.x, y.x, ks[2 * nb], lv[2 * nb]);
                kv::weigh(x.y, y.y, ks[2 * nb + 1], lv[2 * nb + 1]);
            }
        } else {
            // pages of each 8 of these keys (which none of them leaves), and what counts
            int page[2 * KB];
#pragma unroll
            for (int nb = 0; nb < 2 * KB; ++nb) {
                const int at = key + 8 * nb;
                page[nb] = at < k1 ? c.page_of(b, at) : -1;
                if (page[nb] >= 0) bits |= (at + 8 <= k1 ? 255u : (1u << (k1 - at)) - 1u) << (8 * nb);
            }
            if (bits == 0) continue;
#pragma unroll
            for (int nb = 0; nb < 2 * KB; ++nb) {
                const int j = 8 * nb + g;
                const bool on = (bits >> j) & 1u;
                const uint8_t* p = kp + page[nb] * c.k.page + c.slot_of(key + j) * c.k.token;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    ld16(p + 16 * (t + 4 * u), on && PIECE * (t + 4 * u) < a.d, k[nb][u]);
            }
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int j = 16 * kb + 2 * t + (x & 1) + 8 * (x >> 1);
                    const bool on = (bits >> j) & 1u;
                    const uint8_t* p = vp + page[2 * kb + (x >> 1)] * c.v.page + c.slot_of(key + j) * c.v.token;
#pragma unroll
                    for (int w = 0; w < (Q8 ? 0 : HD / 64); ++w)
                        ld16(p + 16 * g + 128 * w, on && 8 * g + 64 * w < a.d, v[kb][x] + 4 * w);
                }
        }
        float s[RP][2 * KB][4];
#pragma unroll
        for (int rp = 0; rp < RP; ++rp)
#pragma unroll
            for (int nb = 0; nb < 2 * KB; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[rp][nb][e] = 0.f;
        constexpr bool pair = RB > 1;
#pragma unroll
        for (int nb = 0; nb < 2 * KB; ++nb)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // the products' second operand: two registers each
                uint32_t w[4 * (Q8 ? 2 : 1)];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    if (Q8)
                        kv::widen4<HELD>(k[nb][u][y], w[2 * y], w[2 * y + (Q8 ? 1 : 0)]);
                    else
                        w[y] = k[nb][u][y];
                }
#pragma unroll
                for (int y = 0; y < (Q8 ? 8 : 4); y += 2)
#pragma unroll
                    for (int rp = 0; rp < RP; ++rp)
                        mma16816<MB>(s[rp][nb], q[2 * rp][u][y], pair ? q[pair ? 2 * rp + 1 : 0][u][y] : 0u,
                                     q[2 * rp][u][y + 1], pair ? q[pair ? 2 * rp + 1 : 0][u][y + 1] : 0u,
                                     w[y], w[y + 1]);
            }
        // Among the tree's keys a row may not see some that others do, and a value of theirs
        // that is not finite would reach it as 0 * NaN: such rows of V are zeroed, and
        // their keys make the rows that see them NaN.
        uint32_t poison = 0;                  // of keys 16 kb + 2 t + (x & 1) + 8 (x >> 1), bit 4 kb + x
        const bool mixed = key + KEYS > ctx;
        if (mixed) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int j = 16 * kb + 2 * t + (x & 1) + 8 * (x >> 1);
                    if (key + j < ctx) continue;
                    bool bad = false;
#pragma unroll
                    for (int w = 0; w < VW; ++w) bad |= nonfinite<HELD, BF>(v[kb][x][w]);
                    poison |= (uint32_t)bad << (4 * kb + x);
                }
            poison |= __shfl_xor_sync(0xffffffffu, poison, 4);
            poison |= __shfl_xor_sync(0xffffffffu, poison, 8);
            poison |= __shfl_xor_sync(0xffffffffu, poison, 16);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (poison >> (4 * kb + x) & 1u) {
#pragma unroll
                        for (int w = 0; w < VW; ++w) v[kb][x][w] = 0;
                    }
        }
        // scores of row 8 rb + g and keys 8 nb + 2 t + {0, 1}
        uint32_t ph[RB][2 * KB], pl[RB][2 * KB];
        float alpha[RB];
        bool moved = false;
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            float x[4 * KB], w[4 * KB], top = -INFINITY;       // (16 bits: w is x)
            const uint32_t sees = bits & (mixed ? tree_window(words[rb], there[rb], key - ctx)
                                                : there[rb] ? 0xffffffffu : 0u);
#pragma unroll
            for (int e = 0; e < 4 * KB; ++e) {
                const int j = 8 * (e >> 1) + 2 * t + (e & 1);
                const float z = s[rb >> 1][e >> 1][2 * (rb & 1) + (e & 1)];
                float y = z * (Q8 ? mul[rb] * ks[e] : mul[rb]);
                // bit 4 kb + x, e = 4 kb + 2 (nb & 1) + (e & 1) and x = (j & 1) + 2 (nb & 1)
                if (poison >> e & 1u) y = __uint_as_float(0x7fc00000u);
                w[e] = (sees >> j) & 1u ? y : -INFINITY;
                x[e] = Q8 ? w[e] + lv[e] : w[e];
                top = fmaxf(top, x[e]);
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            alpha[rb] = 1.f;
            if (top > ref[rb] + 8.f) {
                if (Q8) top = ceilf(top);
                if (ref[rb] != -INFINITY) {
                    alpha[rb] = ex2(ref[rb] - top);
                    sum[rb] = Q8 ? kv::moved_sum(sum[rb], ref[rb] - top) : sum[rb] * alpha[rb];
                }
                ref[rb] = top;
                moved |= alpha[rb] != 1.f;
            }
            const float base = (ref[rb] == -INFINITY ? 0.f : ref[rb]) - kShift;
#pragma unroll
            for (int e = 0; e < 4 * KB; ++e) {
                x[e] = ex2(x[e] - base);
                sum[rb] += Q8 ? ex2(w[e] - base) : x[e];
            }
#pragma unroll
            for (int nb = 0; nb < 2 * KB; ++nb) {
                const uint32_t h = pack16<MB>(x[2 * nb], x[2 * nb + 1]);
                ph[rb][nb] = h;
                if (MB)
                    pl[rb][nb] = pack16<MB>(x[2 * nb] - __uint_as_float(h << 16),
                                            x[2 * nb + 1] - __uint_as_float(h & 0xffff0000u));
            }
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                // O's columns are rows 2 t and 2 t + 1 of the block
                const float a0 = __shfl_sync(0xffffffffu, alpha[rb], 8 * t);
                const float a1 = __shfl_sync(0xffffffffu, alpha[rb], 8 * t + 4);
#pragma unroll
                for (int w = 0; w < NT; ++w) {
                    o[rb][w][0] *= a0;
                    o[rb][w][1] *= a1;
                    o[rb][w][2] *= a0;
                    o[rb][w][3] *= a1;
                }
            }
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                const uint32_t x0 = v[kb][0][w], x1 = v[kb][1][w], x2 = v[kb][2][w], x3 = v[kb][3][w];
                uint32_t m[2][4];             // operands of the products of this register
                if (Q8) {
                    kv::widen4<HELD>(__byte_perm(x0, x1, 0x5140), m[0][0], m[0][1]);
                    kv::widen4<HELD>(__byte_perm(x2, x3, 0x5140), m[0][2], m[0][3]);
                    kv::widen4<HELD>(__byte_perm(x0, x1, 0x7362), m[1][0], m[1][1]);
                    kv::widen4<HELD>(__byte_perm(x2, x3, 0x7362), m[1][2], m[1][3]);
                } else {
                    m[0][0] = __byte_perm(x0, x1, 0x5410);
                    m[0][1] = __byte_perm(x0, x1, 0x7632);
                    m[0][2] = __byte_perm(x2, x3, 0x5410);
                    m[0][3] = __byte_perm(x2, x3, 0x7632);
                }
#pragma unroll
                for (int i = 0; i < (Q8 ? 2 : 1); ++i)
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb) {
                        float* to = o[rb][Q8 ? 2 * w + i : w];
                        mma16816<MB>(to, m[i][0], m[i][1], m[i][2], m[i][3], ph[rb][2 * kb],
                                     ph[rb][2 * kb + 1]);
                        if (MB)
                            mma16816<MB>(to, m[i][0], m[i][1], m[i][2], m[i][3], pl[rb][2 * kb],
                                         pl[rb][2 * kb + 1]);
                    }
            }
    }

    // each warp's rows, then their join
    if (Q8) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        sum[rb] += __shfl_xor_sync(0xffffffffu, sum[rb], 1);
        sum[rb] += __shfl_xor_sync(0xffffffffu, sum[rb], 2);
        if (t == 0) {
            sRef[warp * ROWS + 8 * rb + g] = ref[rb];
            sSum[warp * ROWS + 8 * rb + g] = sum[rb];
        }
#pragma unroll
        for (int w = 0; w < NT; ++w) {
            const int col = Q8 ? HD / 8 * g + 2 * w : 8 * (g + 8 * (w >> 2)) + 2 * (w & 3);
            float* p = sO + warp * kWarpRows + (8 * rb + 2 * t) * HD + col;
            *reinterpret_cast<float2*>(p) = make_float2(o[rb][w][0], o[rb][w][2]);
            *reinterpret_cast<float2*>(p + HD) = make_float2(o[rb][w][1], o[rb][w][3]);
        }
    }
    __syncthreads();
    const int64_t head0 = (int64_t)b * a.H + kh * a.R;
    // the place of a row of the tile among the results, rows (b, head, token)
    const auto place = [&](int row) {
        const int all = group * ROWS + row, tok = all / a.R;
        return (head0 + (all - tok * a.R)) * a.n + tok;
    };
    const auto out_row = [&](int row) {
        const int all = group * ROWS + row, tok = all / a.R;
        return static_cast<T*>(a.o.p) + b * a.o.sb + tok * a.o.st + (int64_t)(kh * a.R + all - tok * a.R) * a.o.sh;
    };
    for (int row = warp; row < nrows; row += kWarps) {
        const int64_t at = place(row);
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sRef[w * ROWS + row]);
        const float base = top == -INFINITY ? 0.f : top;
        float total = 0.f, f[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float by = sRef[w * ROWS + row] - base;
            f[w] = ex2(by);
            total = Q8 ? total + kv::moved_sum(sSum[w * ROWS + row], by) : fmaf(f[w], sSum[w * ROWS + row], total);
        }
        const float inv = total == 0.f ? 0.f : 1.f / total;
        const float lse2 = total == 0.f ? -INFINITY
                           : Q8         ? kv::log_sum(top - kShift, total)
                                        : top - kShift + lg2(total);
        T* out = out_row(row);
        float* part = P.part.out + (split * P.part.rows + at) * a.d;
        for (int e = lane; e < a.d; e += 32) {
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) x = fmaf(f[w], sO[w * kWarpRows + row * HD + e], x);
            x = total == 0.f ? 0.f : x * inv;
            if (P.splits > 1)
                part[e] = x;
            else
                out[e] = from_f<T>(x);
        }
        if (lane == 0) {
            if (P.splits > 1)
                P.part.lse2[split * P.part.rows + at] = lse2;
            else
                a.lse[at] = lse2 * (float)kLn2;
        }
    }
    if (P.splits == 1) return;

    // the last block of these rows joins the splits, in their order
    __threadfence();
    __syncthreads();
    unsigned* count = P.counters + blockIdx.x / P.splits;
    if (threadIdx.x == 0) {
        const unsigned before = atomicAdd(count, 1u);
        sLast = before == (unsigned)P.splits - 1;
        if (sLast) *count = 0;        // ready for the next call
    }
    __syncthreads();
    if (!sLast) return;
    __threadfence();
    // Weights of 256 splits at a time into shared memory (over sO), a row's in one warp;
    // then a thread sums four elements of a row over them.
    constexpr int kSome = 256;
    constexpr int kQuads = HD / 4, kSums = ROWS * kQuads / (32 * kWarps);
    static_assert(ROWS * kSome <= kWarps * kWarpRows, "weights fit over the rows");
    float top[ROWS / kWarps], total[ROWS / kWarps];
#pragma unroll
    for (int x = 0; x < ROWS / kWarps; ++x) {
        const int row = warp + kWarps * x;
        top[x] = -INFINITY;
        total[x] = 0.f;
        if (row < nrows) {
            const float* l = P.part.lse2 + place(row);
            for (int i = lane; i < P.splits; i += 32) top[x] = fmaxf(top[x], l[i * P.part.rows]);
        }
#pragma unroll
        for (int y = 16; y; y >>= 1) top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], y));
    }
    float4 acc[kSums];
#pragma unroll
    for (int x = 0; x < kSums; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < P.splits; s0 += kSome) {
        const int some = min(kSome, P.splits - s0);
        __syncthreads();
#pragma unroll
        for (int x = 0; x < ROWS / kWarps; ++x) {
            const int row = warp + kWarps * x;
            if (row >= nrows) continue;
            const float* l = P.part.lse2 + place(row);
            float w_sum = 0.f;
            for (int i = lane; i < some; i += 32) {
                const float w = ex2(l[(s0 + i) * P.part.rows] - (top[x] == -INFINITY ? 0.f : top[x]));
                sO[row * kSome + i] = w;
                w_sum += w;
            }
#pragma unroll
            for (int y = 16; y; y >>= 1) w_sum += __shfl_xor_sync(0xffffffffu, w_sum, y);
            total[x] += w_sum;
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kSums; ++x) {
            const int e = threadIdx.x + x * 32 * kWarps, row = e / kQuads, col = 4 * (e % kQuads);
            if (row >= nrows || col >= a.d) continue;
            const float* src = P.part.out + (s0 * P.part.rows + place(row)) * a.d + col;
            const float* w = sO + row * kSome;
            const int64_t step = P.part.rows * a.d;
#pragma unroll 16
            for (int i = 0; i < some; ++i) {
                const float4 y = *reinterpret_cast<const float4*>(src + i * step);
                acc[x].x = fmaf(w[i], y.x, acc[x].x);
                acc[x].y = fmaf(w[i], y.y, acc[x].y);
                acc[x].z = fmaf(w[i], y.z, acc[x].z);
                acc[x].w = fmaf(w[i], y.w, acc[x].w);
            }
        }
    }
#pragma unroll
    for (int x = 0; x < ROWS / kWarps; ++x) {
        const int row = warp + kWarps * x;
        if (lane == 0 && row < nrows) {
            sSum[row] = total[x];
            a.lse[place(row)] = total[x] == 0.f ? -INFINITY : (top[x] + lg2(total[x])) * (float)kLn2;
        }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kSums; ++x) {
        const int e = threadIdx.x + x * 32 * kWarps, row = e / kQuads, col = 4 * (e % kQuads);
        if (row >= nrows || col >= a.d) continue;
        T* out = out_row(row) + col;
        const float inv = sSum[row] == 0.f ? 0.f : 1.f / sSum[row];
        const float y[4] = {acc[x].x * inv, acc[x].y * inv, acc[x].z * inv, acc[x].w * inv};
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = from_f<T>(y[i]);
    }
}

// Raises the kernel's limit of shared memory: before its first launch, and before it is asked how
// many blocks an SM holds.
template <int HD, int HELD, bool BF, int RB>
cudaError_t ready() {
    static std::atomic<uint64_t> raised{0};   // devices
    return raise_smem(k_tree_few<HD, HELD, BF, RB>, kFewSmem<HD, HELD, RB>, raised);
}

template <int HD, int HELD, bool BF, int RB>
cudaError_t launch(const FewArgs& p, cudaStream_t s) {
    if (cudaError_t e = ready<HD, HELD, BF, RB>(); e != cudaSuccess) return e;
    const unsigned blocks = (unsigned)((int64_t)p.a.c.B * p.a.c.G * p.groups * p.splits);
    k_tree_few<HD, HELD, BF, RB><<<blocks, 32 * kWarps, kFewSmem<HD, HELD, RB>, s>>>(p);
    count_launch();
    return cudaGetLastError();
}

template <int HD, int HELD, bool BF, int RB>
cudaError_t resident(int* blocks) {
    static std::atomic<int> held{0};
    *blocks = held.load();
    if (*blocks > 0) return cudaSuccess;
    cudaError_t e = ready<HD, HELD, BF, RB>();
    if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, k_tree_few<HD, HELD, BF, RB>, 32 * kWarps,
                                                          kFewSmem<HD, HELD, RB>);
    if (e == cudaSuccess) held.store(*blocks);
    return e;
}

// the kernel of a call, for `f` to run; 16 bits in blocks of 8 rows
template <int HD, int HELD, typename F>
cudaError_t pick_rows(const Args& a, int row_blocks, F f) {
    constexpr int kMost = HELD == HELD_16 ? 1 : 2;
    if (a.bf16)
        return row_blocks == 1 ? f.template run<HD, HELD, true, 1>() : f.template run<HD, HELD, true, kMost>();
    return row_blocks == 1 ? f.template run<HD, HELD, false, 1>() : f.template run<HD, HELD, false, kMost>();
}
template <int HD, typename F>
cudaError_t pick_held(const Args& a, int row_blocks, F f) {
    if (a.c.held == HELD_16) return pick_rows<HD, HELD_16>(a, row_blocks, f);
    return a.c.held == HELD_E4M3 ? pick_rows<HD, HELD_E4M3>(a, row_blocks, f)
                                 : pick_rows<HD, HELD_I8>(a, row_blocks, f);
}
template <typename F>
cudaError_t pick(const Args& a, int row_blocks, F f) {
    return a.d <= 64 ? pick_held<64>(a, row_blocks, f) : pick_held<128>(a, row_blocks, f);
}

struct Launch {
    const FewArgs& p;
    cudaStream_t s;
    template <int HD, int HELD, bool BF, int RB>
    cudaError_t run() const { return launch<HD, HELD, BF, RB>(p, s); }
};
struct Resident {
    int* blocks;
    template <int HD, int HELD, bool BF, int RB>
    cudaError_t run() const { return resident<HD, HELD, BF, RB>(blocks); }
};

}  // namespace

cudaError_t launch_few(const FewArgs& p, cudaStream_t s) { return pick(p.a, p.row_blocks, Launch{p, s}); }

cudaError_t few_resident(const Args& a, int row_blocks, int* blocks) {
    return pick(a, row_blocks, Resident{blocks});
}

}  // namespace tree
}  // namespace fs
