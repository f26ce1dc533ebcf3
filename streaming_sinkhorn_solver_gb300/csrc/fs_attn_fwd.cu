// Cross attention, forward, on the tensor cores.
//
// A block takes 256 queries of one head in two tiles of 128 and streams the
// keys in tiles of 128 (64 for heads wider than 64):
//   S_t = Q_t K^T (TMEM), p = 2^{x - ref} in 16 bits in TMEM,
//   O_t += P_t V (TMEM, P as the A operand read from TMEM).
// V is read as an operand summed over its rows, so nothing is transposed; keys that
// do not count get -inf by one more product (KeyMask), and their rows are zeroed.
//
// Four warps hold a query tile, a row per thread, and one thread issues its
// products, so neither tile waits for the other's.  From the last P of a tile to
// its next scores the tensor core would take its products' time and about 450
// cycles of latency; so P has TMEM columns of its own, and the next scores are
// formed while this tile's are still in the softmax.  That fills TMEM with two S,
// two P and two O for heads up to 64; wider heads take the keys 64 at a time, with
// two P each (their score products then read Q twice as often as keys of 128
// would: 48 cycles of shared memory for 32 of arithmetic, and still less than the
// wait that P in the columns of S costs).
//
// The reference is the running maximum, moved only when a row's maximum grew
// by more than 2^8 (p then stays below 256 times the power of two that
// kProbShift<BF> adds, which the types and the float32 sums hold); the rare move rescales
// O_t in TMEM.  P is rounded to the operands' 16 bits, the sum of p is not: out is 0.22 % off
// in the 2-norm in bfloat16, of which 0.17 % is the rounding of out itself.
//
// Bound: heads of 128 by the products (4 x 4096 x 8192, 16 heads, bfloat16: 720 us,
// 1530 TFLOP/s, 0.81 of the measured burst rate and 0.90 of the sustained one), heads of
// 64 by the softmax (4 x 2048 x 2048, 16 heads: 92 us, 745 TFLOP/s; 16 exponentials a
// cycle and SM, half of what the unit gives, and 47 % of the issue slots).
#include "fs_attn_host.cuh"

#include <atomic>
#include <type_traits>

namespace fs {
namespace attn {

namespace {

constexpr int kSoftWarps = 8;              // 4 per query tile
constexpr int kFwdThreads = 32 * (kSoftWarps + 4);
constexpr int kMma0 = kSoftWarps, kLoad = kSoftWarps + 2, kClean = kSoftWarps + 3;
constexpr int kSlack = 2 * kTile;          // bias table entries beyond +-D on each side
constexpr float kRefSlack = 8.f;

// Key tiles, TMEM columns and shared memory by the width of the heads
template <int HD>
struct Fwd {
    static constexpr int kChunks = HD / 64;
    static constexpr int kKeys = forward_keys(HD);               // keys of a tile
    static constexpr int kChunkBytes = kKeys * 128;              // 64 elements of each
    static constexpr int kTileBytes = kChunks * kChunkBytes;     // 16 KB
    static constexpr int kQBytes = kChunks * CHUNK_BYTES;
    static constexpr int kStages = 8;                            // K and V tiles in turn
    static constexpr int kPBufs = HD == 64 ? 1 : 2;
    static constexpr uint32_t kPCols = kKeys / 2;
    __host__ __device__ static constexpr uint32_t S(int t) { return 256 * t; }
    __host__ __device__ static constexpr uint32_t P(int t) { return S(t) + kKeys; }
    __host__ __device__ static constexpr uint32_t O(int t) { return P(t) + kPBufs * kPCols; }
    static_assert(kKeys + kPBufs * (int)kPCols + HD == 256, "TMEM");
};

struct FwdBars {
    uint64_t full[8], empty[8], clean[8], last[2];
    uint64_t qfull, sfull[2], sfree[2], pfull[2][2], pfree[2][2], drain[2];
    uint32_t tmem, pad;
};
template <int HD>
using FwdMask = KeyMask<Fwd<HD>::kKeys, Fwd<HD>::kStages / 2>;
template <int HD>
constexpr size_t kFwdFixed = 1024 + 2 * (size_t)Fwd<HD>::kQBytes + Fwd<HD>::kStages * (size_t)Fwd<HD>::kTileBytes +
                             FwdMask<HD>::kBytes + sizeof(FwdBars);

// MASK: tiles may hold keys that do not count
template <int HD, bool BF, bool MASK>
__global__ void __launch_bounds__(kFwdThreads, 1) k_forward_tc(const __grid_constant__ FwdArgs P) {
    using C = Fwd<HD>;
    using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    constexpr int NS = C::kStages, KT = C::kKeys;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    const Args& a = P.a;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    uint8_t* sQ = smem;                                  // at the end the rows of out
    uint8_t* sKV = sQ + 2 * C::kQBytes;
    const FwdMask<HD> mask{sKV + NS * C::kTileBytes};
    FwdBars& bar = *reinterpret_cast<FwdBars*>(mask.p + FwdMask<HD>::kBytes);
    float* sBias = reinterpret_cast<float*>(&bar + 1);

    int blk = blockIdx.x;
    const int split = blk % P.splits;
    blk /= P.splits;
    const int qt = blk % P.row_blocks;
    blk /= P.row_blocks;
    const int h = blk % a.H;
    const int b = longest_first<KT>(P.kt, a, blk / a.H);
    const int i0 = qt * 2 * kTile;
    const bool two = i0 + kTile < a.n;
    const int end = key_end(a, b);
    const int nt_all = step_count<KT>(P.kt, b, end);
    const int per = (nt_all + P.splits - 1) / P.splits;
    const int t0 = min(nt_all, split * per);
    const int nt = min(nt_all, t0 + per) - t0;
    const int dsteps = (a.d + 15) >> 4;
    // Tiles with keys that do not count are waited for at their cleaning.  Under a mask
    // any tile may be one; else the one that the keys end in, whose copies have barriers
    // of their own (the cleaning warp then follows no other tile's).
    const bool every = MASK && P.kt.words;
    const int tail = MASK && !every && (t0 + nt) * KT > end ? nt - 1 : nt;

    // The loading warp's barriers are its own until the block meets below: it starts
    // its copies before that.
    if (warp == kLoad) {
        if (lane < NS) mbar_init(&bar.full[lane], 1);
        if (lane == NS) mbar_init(&bar.qfull, 1);
        if (lane > NS && lane <= NS + 2) mbar_init(&bar.last[lane - NS - 1], 1);
        fence_mbar_init();
        __syncwarp();
    } else if (warp == kClean) {
        if (lane < NS) {
            mbar_init(&bar.empty[lane], two ? 2 : 1);
            mbar_init(&bar.clean[lane], 1);
        } else if (lane < NS + 2) {
            const int t = lane - NS;
            mbar_init(&bar.sfull[t], 1);
            mbar_init(&bar.sfree[t], 4);
            mbar_init(&bar.pfull[t][0], 4);
            mbar_init(&bar.pfull[t][1], 4);
            mbar_init(&bar.pfree[t][0], 1);
            mbar_init(&bar.pfree[t][1], 1);
            mbar_init(&bar.drain[t], 1);
        }
        fence_mbar_init();
    }
    if (warp == kMma0) tmem_alloc(&bar.tmem, 512);
    // the copy of step it (K and V in turn) into its slot
    const auto load = [&](int it, int slot) {
        uint64_t* const full = (it >> 1) == tail ? &bar.last[it & 1] : &bar.full[slot];
        const int g = h / a.R;
        const int key = step_key<KT>(P.kt, b, t0 + (it >> 1));
        const TensorMap& src = it & 1 ? P.v : P.k;
        mbar_arrive_expect_tx(full, C::kTileBytes);
        for (int c = 0; c < C::kChunks; ++c)
            tma_load(sKV + slot * C::kTileBytes + c * C::kChunkBytes, &src.map, c * 64, key, g * src.head,
                     b * src.batch, full);
    };
    const int early = min(2 * nt, NS);     // copies that need no free slot
    if (warp == kLoad && nt > 0 && elect_one()) {
        mbar_arrive_expect_tx(&bar.qfull, (two ? 2 : 1) * C::kQBytes);
        for (int t = 0; t < (two ? 2 : 1); ++t)
            for (int c = 0; c < C::kChunks; ++c)
                tma_load(sQ + t * C::kQBytes + c * CHUNK_BYTES, &P.q.map, c * 64, i0 + t * kTile,
                         h * P.q.head, b * P.q.batch, &bar.qfull);
        for (int it = 0; it < early; ++it) load(it, it);
    }
    if (a.table) {
        // base-2 bias by relative position -D - kSlack .. D + kSlack of this head
        const T* row = static_cast<const T*>(a.table) + h * a.table_stride;
#pragma unroll 4      // two loads that depend on one another an entry
        for (int e = threadIdx.x; e < 2 * (a.D + kSlack) + 1; e += kFwdThreads)
            sBias[e] = bias2(to_f<T>(row[bucket_of(a, (int64_t)e - a.D - kSlack)]));
    }
    if (MASK) mask.init(threadIdx.x, kFwdThreads);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;

    if (warp == kLoad) {
        if (nt > 0 && elect_one()) {
            Ring r;
            r.step(early, NS);
            int issued = early;
            bool ok = true;
            for (int it = early; it < 2 * nt; ++it) {
                if (!mbar_wait(&bar.empty[r.slot], r.phase ^ 1u, a.err, ERR_TIMEOUT_PRODUCER)) {
                    ok = false;
                    break;
                }
                load(it, r.slot);
                ++issued;
                r.step(1, NS);
            }
            if (!ok) {   // every copy lands before the block can exit
                mbar_wait(&bar.qfull, 0, a.err, ERR_TIMEOUT_PRODUCER);
                Ring l;
                for (int it = 0; it < issued; ++it) {
                    if ((it >> 1) == tail)
                        mbar_wait(&bar.last[it & 1], 0, a.err, ERR_TIMEOUT_PRODUCER);
                    else if (it + NS >= issued)
                        mbar_wait(&bar.full[l.slot], l.phase, a.err, ERR_TIMEOUT_PRODUCER);
                    l.step(1, NS);
                }
            }
        }
    } else if (warp == kMma0 || warp == kMma0 + 1) {
        const int t = warp - kMma0;
        if (nt > 0 && (t == 0 || two) && elect_one()) {
            const uint32_t idS = idesc_16(BF, KT, false), idM = idesc_16(true, KT, false);
            const uint32_t idO = idesc_16(BF, dsteps * 16, true);
            constexpr uint64_t kTileU = C::kTileBytes >> 4;    // descriptors count 16 bytes
            const uint64_t dQ = sdesc_sw128(smem_u32(sQ)) + t * (C::kQBytes >> 4);
            const uint64_t dK = sdesc_sw128(smem_u32(sKV));
            const uint64_t dV = sdesc_tokens(smem_u32(sKV), C::kChunkBytes);
            const uint32_t cS = tmem + C::S(t), cP = tmem + C::P(t), cO = tmem + C::O(t);
            uint64_t* const kvbar = every ? bar.clean : bar.full;
            const auto landed = [&](const Ring& r, int j) {
                return mma_wait(a.err, (MASK && j == tail ? bar.clean : kvbar) + r.slot,
                                MASK && j == tail ? 0 : r.phase);
            };
            const uint64_t dOnes = mask.ones(), dMask = mask.tile(0);
            Ring rk, rv;
            rv.step(1, NS);
            bool ok = mma_wait(a.err, &bar.qfull, 0);
            for (int j = -1; j < nt && ok; ++j) {
                if (j + 1 < nt) {
                    if (!(ok = landed(rk, j + 1) &&
                               (j < 0 || mma_wait(a.err, &bar.sfree[t], j & 1))))
                        break;
                    mma_over_d<4, C::kChunkBytes>(cS, dQ, dK + rk.slot * kTileU, idS, (dsteps + 3) / 4);
                    if (MASK) {
                        const uint64_t dTile = dMask + (rk.slot >> 1) * FwdMask<HD>::kStep;
                        const int times = every || j + 1 == tail;     // a loop bound (mma_over_d)
#pragma unroll 1
                        for (int x = 0; x < times; ++x) mma_f16(cS, dOnes, dTile, idM, true);
                    }
                    mma_commit(&bar.sfull[t]);
                    mma_commit(&bar.empty[rk.slot]);
                    rk.step(2, NS);
                }
                if (j < 0) continue;
                const int buf = C::kPBufs == 2 ? j & 1 : 0;
                if (!(ok = landed(rv, j) &&
                           mma_wait(a.err, &bar.pfull[t][buf], C::kPBufs == 2 ? (j >> 1) & 1 : j & 1)))
                    break;
                mma_over_tokens<KT>(cO, cP + buf * C::kPCols, dV + rv.slot * kTileU, idO, j > 0, 32);
                mma_commit(&bar.pfree[t][buf]);
                mma_commit(&bar.empty[rv.slot]);
                rv.step(2, NS);
            }
            mma_commit(&bar.drain[t]);
            mbar_wait(&bar.drain[t], 0, a.err, ERR_TIMEOUT_MMA);
        }
    } else if (warp == kClean) {
        if (MASK && nt > 0) {
            const int j0 = every ? 0 : tail;
            Ring r;
            r.slot = 2 * j0 % NS;
            bool ok = true;
            KeyBits<KT> next(P.kt, b, t0 + min(j0, nt - 1), end);
            for (int j = j0; j < nt && ok; ++j) {
                const KeyBits<KT> w = next;
                if (j + 1 < nt) next = KeyBits<KT>(P.kt, b, t0 + j + 1, end);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    ok = ok && warp_wait(every ? &bar.full[r.slot] : &bar.last[kv], r.phase, a.err,
                                         ERR_TIMEOUT_PRODUCER);
                    if (!ok) break;
                    if (!kv) mask.write(r.slot >> 1, w, lane);
                    clear_rows(sKV + r.slot * C::kTileBytes, C::kChunks, C::kChunkBytes, w, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.clean[r.slot]);
                    r.step(1, NS);
                }
            }
        }
    } else {
        const int t = warp >> 2, quarter = warp & 3;
        if (t == 0 || two) {
            const int r = quarter * 32 + lane;
            const int i = i0 + t * kTile + r;
            const uint32_t lofs = (uint32_t)(quarter * 32) << 16;
            const uint32_t tS = tmem + C::S(t) + lofs, tP = tmem + C::P(t) + lofs, tO = tmem + C::O(t) + lofs;
            // position of the tile's first query
            const int64_t first = (a.q_pos ? (int64_t)__ldg(a.q_pos + b) : 0) + i0 + t * kTile;
            float ref = -INFINITY, sum = 0.f;
            bool ok = true;
            for (int j = 0; j < nt; ++j) {
                if (!(ok = warp_wait(&bar.sfull[t], j & 1, a.err, ERR_TIMEOUT_EPILOGUE))) break;
                tc_fence_after();
                float v[KT];
#pragma unroll
                for (int c = 0; c < KT; c += 32) tmem_ld32(tS + c, v + c);
                tmem_wait_ld();
                tmem_reg_fence(v);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.sfree[t]);
                float mul = a.scale2, add = 0.f;
                if (a.table) {
                    // relative position of the first row and key
                    const int64_t rel0 = step_key<KT>(P.kt, b, t0 + j) - first;
                    if (rel0 - (kTile - 1) >= a.D) {
                        add = sBias[2 * a.D + kSlack];
                    } else if (rel0 + (KT - 1) <= -a.D) {
                        add = sBias[kSlack];
                    } else {
                        // |rel| < D + 2 * 128 here
                        const float* e = sBias + (int)rel0 - r + a.D + kSlack;
#pragma unroll
                        for (int c = 0; c < KT; ++c) v[c] = fmaf(v[c], mul, e[c]);
                        mul = 1.f;
                    }
                }
                float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                for (int c = 4; c + 8 <= KT; c += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k) m[k] = max3(m[k], v[c + 2 * k], v[c + 2 * k + 1]);
                m[0] = max3(m[0], v[KT - 4], v[KT - 3]);
                m[1] = max3(m[1], v[KT - 2], v[KT - 1]);
                const float top = fmaf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), mul, add);
                float alpha = 1.f;
                if (top > ref + kRefSlack) {
                    // (up to its first counted key a row's sum and O are zero)
                    if (ref != -INFINITY) alpha = ex2(ref - top);
                    sum *= alpha;
                    ref = top;
                }
                const int buf = C::kPBufs == 2 ? j & 1 : 0;
                if (__any_sync(0xffffffffu, alpha != 1.f)) {
                    // O is still once the products of tile j - 1 are done (j > 0 here)
                    if (!(ok = warp_wait(&bar.pfree[t][C::kPBufs == 2 ? buf ^ 1 : 0],
                                         C::kPBufs == 2 ? ((j - 1) >> 1) & 1 : (j - 1) & 1, a.err,
                                         ERR_TIMEOUT_EPILOGUE)))
                        break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < dsteps * 16; c += 16) {
                        float o[16];
                        tmem_ld16(tO + c, o);
                        tmem_wait_ld();
                        tmem_reg_fence(o);
                        uint32_t u[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * alpha);
                        tmem_st16(tO + c, u);
                    }
                }
                const float base = add + kProbShift<BF> - (ref == -INFINITY ? 0.f : ref);
                const uint64_t mul2 = pk(mul, mul), base2 = pk(base, base);
                uint64_t s0 = 0, s1 = 0;
#pragma unroll
                for (int q = 0; q < KT / 64; ++q) {
                    uint32_t p[32];
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const int x = q * 64 + 2 * c;
                        float e0, e1, e2, e3;
                        upk(fma2(pk(v[x], v[x + 1]), mul2, base2), e0, e1);
                        upk(fma2(pk(v[x + 2], v[x + 3]), mul2, base2), e2, e3);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        e2 = ex2(e2);
                        e3 = ex2(e3);
                        s0 = add2(s0, pk(e0, e1));
                        s1 = add2(s1, pk(e2, e3));
                        p[c] = pack16<BF>(e0, e1);
                        p[c + 1] = pack16<BF>(e2, e3);
                    }
                    // the buffer's last P has been read: of two, the one of tile j - 2 was when
                    // S of this tile was done (its products were issued before it)
                    if (q == 0 && j > 0 && C::kPBufs == 1) {
                        ok = warp_wait(&bar.pfree[t][0], (j - 1) & 1, a.err, ERR_TIMEOUT_EPILOGUE);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    tmem_st32(tP + buf * C::kPCols + q * 32, p);
                }
                if (!ok) break;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.pfull[t][buf]);
                float f0, f1, f2, f3;
                upk(s0, f0, f1);
                upk(s1, f2, f3);
                sum += (f0 + f1) + (f2 + f3);
            }
            if (nt > 0 && ok) {
                const int j = nt - 1;
                ok = warp_wait(&bar.pfree[t][C::kPBufs == 2 ? j & 1 : 0],
                               C::kPBufs == 2 ? (j >> 1) & 1 : j & 1, a.err, ERR_TIMEOUT_EPILOGUE);
            }
            const bool live = i < a.n;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int64_t row = ((int64_t)b * a.H + h) * a.n + i;
            if (live) {
                const float lse2 = sum == 0.f ? -INFINITY : ref - kProbShift<BF> + lg2(sum);
                if (P.splits > 1)
                    P.part.lse2[split * P.part.rows + row] = lse2;
                else
                    a.lse[row] = lse2 * (float)kLn2;
            }
            tc_fence_after();
            // the rows of out, through this warp's rows of the tile's Q
            float* part = P.splits > 1 ? P.part.out + (split * P.part.rows + row) * a.d : nullptr;
            uint8_t* stage = sQ + t * C::kQBytes;
#pragma unroll 2
            for (int c = 0; c < dsteps * 16 && ok; c += 16) {
                float o[16];
                if (nt > 0) {
                    tmem_ld16(tO + c, o);
                    tmem_wait_ld();
                    tmem_reg_fence(o);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = sum == 0.f ? 0.f : o[e] * inv;
                if (part) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (live && c + e < a.d) part[c + e] = o[e];
                    __syncwarp();
                } else {
                    stage16<BF>(stage, r, c, o);
                }
            }
            if (!part) {
                const int w0 = i - lane;      // the warp's first query
                unstage_rows<32>(stage, quarter * 32, a.n - w0, a.d,
                             static_cast<uint16_t*>(a.o.p) + b * a.o.sb + (int64_t)w0 * a.o.st + h * a.o.sh,
                             a.o.st, P.out_vec, lane);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMma0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int HD, bool BF, bool MASK>
cudaError_t launch_masked(const FwdArgs& p, cudaStream_t s) {
    const size_t bias = p.a.table ? sizeof(float) * (2 * (size_t)(p.a.D + kSlack) + 1) : 0;
    constexpr size_t most = kFwdFixed<HD> + sizeof(float) * (2 * (size_t)(kMaxDistance + kSlack) + 1);
    static_assert(most <= kSmemLimit, "forward kernel does not fit in shared memory");
    static std::atomic<uint64_t> ready{0};    // devices whose shared-memory limit is raised
    if (cudaError_t e = raise_smem(k_forward_tc<HD, BF, MASK>, most, ready); e != cudaSuccess) return e;
    const unsigned blocks = (unsigned)((int64_t)p.row_blocks * p.a.H * p.a.B * p.splits);
    k_forward_tc<HD, BF, MASK><<<blocks, kFwdThreads, kFwdFixed<HD> + bias, s>>>(p);
    count_launch();
    return cudaGetLastError();
}

template <int HD, bool BF>
cudaError_t launch_forward(const FwdArgs& p, cudaStream_t s) {
    const bool whole = !p.kt.words && !p.a.kv_len && p.a.m % Fwd<HD>::kKeys == 0;
    return whole ? launch_masked<HD, BF, false>(p, s) : launch_masked<HD, BF, true>(p, s);
}

}  // namespace

cudaError_t launch_forward_tc(const FwdArgs& p, cudaStream_t s) {
    if (p.a.d <= 64)
        return p.a.bf16 ? launch_forward<64, true>(p, s) : launch_forward<64, false>(p, s);
    return p.a.bf16 ? launch_forward<128, true>(p, s) : launch_forward<128, false>(p, s);
}

}  // namespace attn
}  // namespace fs
