// Cross attention, gradients, on the tensor cores.  Two kernels, because the
// results are sums over different axes and no float atomics are used (results
// are bitwise repeatable): the scores are formed in both, seven products where
// five are needed.
//
// k_grad_q: a block takes 128 queries of one head and streams the keys.
//     S = Q K^T, dP = dO V^T, p = 2^{x - lse2}, ds = p (dP - delta),
//     dQ += ds K;   Q and dO stay in TMEM as the A operands of S and dP, ds
//     replaces dP there as the A operand of dQ.
//   Also delta_i = dO_i . O_i, the padded rows (lse2, delta) that k_grad_kv
//   reads, and the sums of ds by relative position for the bias gradient.
// k_grad_kv: a block takes 128 keys of one key head and streams the queries of
//   all its heads, with keys as rows:
//     S = K Q^T, dP = V dO^T, dV += p dO, dK += ds Q;   p replaces S in TMEM
//     and ds replaces dP, each the A operand of its product.
// In both, eight warps hold the elementwise part: warps w and w + 4 the same 32
// rows, 64 columns each; one thread issues the products in an order that keeps
// the tensor core at the next tile's scores while this tile's are in registers.
#include "fs_attn_host.cuh"

#include <atomic>
#include <type_traits>

namespace fs {
namespace attn {

namespace {

constexpr int kGradThreads = 384;
constexpr int kSlack = 2 * kTile;
constexpr int kMaxRing = 8;
constexpr int kElemWarps = 8;
constexpr int kBands = 4;           // rows of bias sums: one per 32 queries

// barriers, then the TMEM address
struct GradBars {
    uint64_t full[kMaxRing], empty[kMaxRing], clean[kMaxRing];
    uint64_t ready, sfull, sfree, done, drain, pfull, dsfull;
    uint64_t dpfull[2];
    uint32_t tmem, pad;
};

template <bool BF>
using Elem = typename std::conditional<BF, __nv_bfloat16, __half>::type;

// Two 16-bit values of a register as floats
template <bool BF>
__device__ __forceinline__ float2 unpack16(uint32_t u) {
    if (BF) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    const __half2 h = *reinterpret_cast<__half2*>(&u);
    return __half22float2(h);
}

// The row's elements [c, c + 16) as 8 registers, zero beyond d; `vec`: 16-byte loads
template <bool BF>
__device__ __forceinline__ void load16(const View& w, int64_t off, int c, int d, bool live, bool vec,
                                       uint32_t* u) {
    const uint16_t* p = static_cast<const uint16_t*>(w.p) + off;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (live && vec) {
            if (c + 8 * e < d) x = __ldg(reinterpret_cast<const uint4*>(p + c + 8 * e));
        } else if (live) {
            uint32_t* xs = &x.x;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c + 8 * e + k < d) xs[k >> 1] |= (uint32_t)__ldg(p + c + 8 * e + k) << (16 * (k & 1));
        }
        u[4 * e] = x.x;
        u[4 * e + 1] = x.y;
        u[4 * e + 2] = x.z;
        u[4 * e + 3] = x.w;
    }
}

// Columns [c0, c1) of a row of sums in TMEM, times `mul`, rounded, to a row in memory
// (zero where !keep).  Whole warps.
template <bool BF>
__device__ __forceinline__ void store_row(const View& w, int64_t off, uint32_t tmem_row, int c0, int c1,
                                          int d, float mul, bool any, bool live, bool keep, bool vec) {
    using T = Elem<BF>;
    T* out = static_cast<T*>(w.p) + off;
    for (int c = c0; c < c1; c += 16) {
        float o[16];
        if (any) {
            tmem_ld16(tmem_row + c, o);
            tmem_wait_ld();
            tmem_reg_fence(o);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = any && keep ? o[e] * mul : 0.f;
        if (vec) {
#pragma unroll
            for (int e = 0; e < 16; e += 8)
                if (live && c + e < d)
                    *reinterpret_cast<uint4*>(out + c + e) =
                        make_uint4(pack16<BF>(o[e], o[e + 1]), pack16<BF>(o[e + 2], o[e + 3]),
                                   pack16<BF>(o[e + 4], o[e + 5]), pack16<BF>(o[e + 6], o[e + 7]));
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (live && c + e < d) out[c + e] = from_f<T>(o[e]);
        }
        __syncwarp();
    }
}

// base-2 bias of head h by relative position -D - kSlack .. D + kSlack
template <bool BF>
__device__ __forceinline__ void fill_bias(const Args& a, int h, float* sBias, int t, int threads) {
    const Elem<BF>* row = static_cast<const Elem<BF>*>(a.table) + h * a.table_stride;
    for (int e = t; e < 2 * (a.D + kSlack) + 1; e += threads)
        sBias[e] = bias2(to_f<Elem<BF>>(row[bucket_of(a, (int64_t)e - a.D - kSlack)]));
}

// ---------------------------------------------------------------------------

// TMEM columns of k_grad_q.  ds of tile j replaces dP of tile j; with heads of 64
// there is room for two dP tiles, so the next one does not wait for dQ.
template <int HD>
struct QCols {
    static constexpr int kDp = HD == 64 ? 2 : 1;
    static constexpr uint32_t S = 0, DP = kTile, DQ = DP + kDp * kTile, Q = DQ + HD, DO = Q + HD / 2;
    static_assert(DO + HD / 2 <= 512, "TMEM");
};

template <int HD, bool BF>
__global__ void __launch_bounds__(kGradThreads, 1) k_grad_q(const __grid_constant__ GradArgs P) {
    using Cols = QCols<HD>;
    constexpr int kChunks = HD / 64, kTileBytes = kChunks * CHUNK_BYTES;
    constexpr uint64_t kTileU = kTileBytes >> 4;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    const Args& a = P.a;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int NS = P.stages;
    uint8_t* sKV = smem;
    GradBars& bar = *reinterpret_cast<GradBars*>(sKV + NS * kTileBytes);
    float* sDelta = reinterpret_cast<float*>(&bar + 1);          // [128]
    float* sFar = sDelta + kTile;                                // [8][2]
    float* sBias = sFar + 2 * kElemWarps;                        // [2 (D + kSlack) + 1]
    float* sSums = sBias + (a.table ? 2 * (a.D + kSlack) + 1 : 0);   // [4][2 D + 1]

    int blk = blockIdx.x;
    const int qt = blk % P.q_tiles;
    blk /= P.q_tiles;
    const int h = blk % a.H;
    const int b = blk / a.H;
    const int i0 = qt * kTile;
    const int end = key_end(a, b);
    const int nt = tile_count(P.kt, b, end);
    const bool partial_keys = P.kt.words != nullptr || end < a.m;
    const int64_t first = (a.q_pos ? (int64_t)__ldg(a.q_pos + b) : 0) + i0;
    const int dsteps = (a.d + 15) >> 4;
    const int width = 2 * a.D + 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&bar.full[s], 1);
            mbar_init(&bar.empty[s], 1);
            mbar_init(&bar.clean[s], 1);
        }
        mbar_init(&bar.ready, kElemWarps);
        mbar_init(&bar.sfull, 1);
        mbar_init(&bar.sfree, kElemWarps);
        mbar_init(&bar.dpfull[0], 1);
        mbar_init(&bar.dpfull[1], 1);
        mbar_init(&bar.dsfull, kElemWarps);
        mbar_init(&bar.done, 1);
        mbar_init(&bar.drain, 1);
        fence_mbar_init();
    }
    if (warp == 9) tmem_alloc(&bar.tmem, 512);
    if (a.table) fill_bias<BF>(a, h, sBias, threadIdx.x, kGradThreads);
    if (a.bias_part)
        for (int e = threadIdx.x; e < 4 * width; e += kGradThreads) sSums[e] = 0.f;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;

    if (warp == 8) {
        if (nt > 0 && elect_one()) {
            const int g = h / a.R;
            Ring r;
            int issued = 0;
            bool ok = true;
            for (int it = 0; it < 2 * nt; ++it) {
                if (!mbar_wait(&bar.empty[r.slot], r.phase ^ 1u, a.err, ERR_TIMEOUT_PRODUCER)) {
                    ok = false;
                    break;
                }
                const int tile = tile_at(P.kt, b, it >> 1);
                const TensorMap& src = it & 1 ? P.v : P.k;
                mbar_arrive_expect_tx(&bar.full[r.slot], kTileBytes);
                for (int c = 0; c < kChunks; ++c)
                    tma_load(sKV + r.slot * kTileBytes + c * CHUNK_BYTES, &src.map, c * 64, tile * kTile,
                             g * src.head, b * src.batch, &bar.full[r.slot]);
                ++issued;
                r.step(1, NS);
            }
            if (!ok) {   // every copy lands before the block can exit
                Ring l;
                for (int it = 0; it < issued; ++it) {
                    if (it + NS >= issued)
                        mbar_wait(&bar.full[l.slot], l.phase, a.err, ERR_TIMEOUT_PRODUCER);
                    l.step(1, NS);
                }
            }
        }
    } else if (warp == 9) {
        if (nt > 0 && elect_one()) {
            const uint32_t idS = idesc_16(BF, kTile, false);
            const uint32_t idQ = idesc_16(BF, dsteps * 16, true);
            const uint64_t dKV = sdesc_sw128(smem_u32(sKV)), dKVt = sdesc_tokens(smem_u32(sKV));
            Ring rk, rv, rq;     // K of the next scores, V of the next dP, K of the next dQ
            rv.step(1, NS);
            uint64_t* kbar = partial_keys ? bar.clean : bar.full;
            bool ok = mma_wait(a.err, &bar.ready, 0) && mma_wait(a.err, &kbar[rk.slot], rk.phase);
            if (ok) {
                mma_over_d_ts(tmem + Cols::S, tmem + Cols::Q, dKV + rk.slot * kTileU, idS, dsteps);
                mma_commit(&bar.sfull);
                rk.step(2, NS);
                ok = mma_wait(a.err, &bar.full[rv.slot], rv.phase);
            }
            if (ok) {
                mma_over_d_ts(tmem + Cols::DP, tmem + Cols::DO, dKV + rv.slot * kTileU, idS, dsteps);
                mma_commit(&bar.dpfull[0]);
                mma_commit(&bar.empty[rv.slot]);
                rv.step(2, NS);
            }
            for (int j = 0; j < nt && ok; ++j) {
                const bool more = j + 1 < nt;
                const uint32_t next = Cols::kDp == 2 ? (j + 1) & 1 : 0;
                if (more) {
                    // scores of the next tile, once this one's are in registers
                    if (!(ok = mma_wait(a.err, &kbar[rk.slot], rk.phase) && mma_wait(a.err, &bar.sfree, j & 1))) break;
                    mma_over_d_ts(tmem + Cols::S, tmem + Cols::Q, dKV + rk.slot * kTileU, idS, dsteps);
                    mma_commit(&bar.sfull);
                    rk.step(2, NS);
                }
                if (more && Cols::kDp == 2) {
                    if (!(ok = mma_wait(a.err, &bar.full[rv.slot], rv.phase))) break;
                    mma_over_d_ts(tmem + Cols::DP + next * kTile, tmem + Cols::DO, dKV + rv.slot * kTileU,
                                  idS, dsteps);
                    mma_commit(&bar.dpfull[next]);
                    mma_commit(&bar.empty[rv.slot]);
                    rv.step(2, NS);
                }
                if (!(ok = mma_wait(a.err, &bar.dsfull, j & 1))) break;
                mma_over_tokens(tmem + Cols::DQ, tmem + Cols::DP + (Cols::kDp == 2 ? (j & 1) * kTile : 0),
                                dKVt + rq.slot * kTileU, idQ, j > 0, 64);
                mma_commit(&bar.empty[rq.slot]);
                rq.step(2, NS);
                if (more && Cols::kDp == 1) {
                    if (!(ok = mma_wait(a.err, &bar.full[rv.slot], rv.phase))) break;
                    mma_over_d_ts(tmem + Cols::DP, tmem + Cols::DO, dKV + rv.slot * kTileU, idS, dsteps);
                    mma_commit(&bar.dpfull[0]);
                    mma_commit(&bar.empty[rv.slot]);
                    rv.step(2, NS);
                }
            }
            mma_commit(&bar.done);
            mma_commit(&bar.drain);
            mbar_wait(&bar.drain, 0, a.err, ERR_TIMEOUT_MMA);
        }
    } else if (warp == 10) {
        if (partial_keys) {
            Ring r;
            for (int j = 0; j < nt; ++j) {
                const KeyBits<kTile> w(P.kt, b, j, end);
                if (!warp_wait(&bar.full[r.slot], r.phase, a.err, ERR_TIMEOUT_PRODUCER)) break;
                if (!w.all()) {
                    clear_rows(sKV + r.slot * kTileBytes, kChunks, CHUNK_BYTES, w, lane);
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.clean[r.slot]);
                r.step(2, NS);
            }
        }
    } else if (warp < kElemWarps) {
        const int quarter = warp & 3, half = warp >> 2;
        const int r = quarter * 32 + lane;
        const int i = i0 + r;
        const bool live = i < a.n;
        const uint32_t lofs = (uint32_t)(quarter * 32) << 16;
        const int64_t row = ((int64_t)b * a.H + h) * a.n + i;
        // operands into TMEM: warps 0..3 the rows of Q, warps 4..7 those of dO with delta
        {
            const View& w = half ? a.dout : a.q;
            const int64_t off = b * w.sb + (int64_t)i * w.st + h * w.sh;
            const int64_t oo = b * a.o.sb + (int64_t)i * a.o.st + h * a.o.sh;
            float dot = 0.f;
            for (int x = 0; x < dsteps; ++x) {
                uint32_t u[8];
                load16<BF>(w, off, 16 * x, a.d, live, half ? P.dout_vec : P.q_vec, u);
                if (half) {
                    uint32_t v[8];
                    load16<BF>(a.o, oo, 16 * x, a.d, live, P.o_vec, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 f = unpack16<BF>(u[e]), g = unpack16<BF>(v[e]);
                        dot = fmaf(f.x, g.x, dot);
                        dot = fmaf(f.y, g.y, dot);
                    }
                }
                __syncwarp();
                tmem_st8u(tmem + lofs + (half ? Cols::DO : Cols::Q) + 8 * x, u);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.ready);
            if (half) sDelta[r] = dot;
        }
        // a row without a counted key has p = 0, as if its lse were +inf
        float lse2 = live ? a.lse[row] * (float)kLog2e : INFINITY;
        if (lse2 == -INFINITY) lse2 = INFINITY;
        named_sync(1, 32 * kElemWarps);
        const float delta = sDelta[r];
        if (half == 0) {
            float* pad = P.rows + (((int64_t)b * a.H + h) * P.q_tiles + qt) * 2 * kTile;
            pad[r] = -lse2;
            pad[kTile + r] = delta;
        }
        const float nlse = -lse2;
        float far_lo = 0.f, far_hi = 0.f;
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            const int tile = tile_at(P.kt, b, j);
            const uint4 w = tile_words(P.kt, b, tile, end);
            // relative position of the warp's first row and column
            const int64_t rel0 = (int64_t)tile * kTile + half * 64 - first - quarter * 32;
            const int buf = Cols::kDp == 2 ? j & 1 : 0;
            if (!(ok = warp_wait(&bar.sfull, j & 1, a.err, ERR_TIMEOUT_EPILOGUE))) break;
            tc_fence_after();
            float v[64];
            tmem_ld32(tmem + lofs + Cols::S + half * 64, v);
            tmem_ld32(tmem + lofs + Cols::S + half * 64 + 32, v + 32);
            tmem_wait_ld();
            tmem_reg_fence(v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.sfree);
            float mul = a.scale2, add = 0.f;
            int where = 0;                       // -1, 1: every pair beyond -D or D
            if (a.table) {
                if (rel0 - 31 >= a.D) {
                    add = sBias[2 * a.D + kSlack];
                    where = 1;
                } else if (rel0 + 63 <= -a.D) {
                    add = sBias[kSlack];
                    where = -1;
                } else {
                    const float* e = sBias + (int)rel0 - lane + a.D + kSlack;
#pragma unroll
                    for (int c = 0; c < 64; ++c) v[c] = fmaf(v[c], mul, e[c]);
                    mul = 1.f;
                }
            }
            const float base = add + nlse;
            const uint64_t mul2 = pk(mul, mul), base2 = pk(base, base);
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
                upk(fma2(pk(v[c], v[c + 1]), mul2, base2), v[c], v[c + 1]);
                v[c] = ex2(v[c]);
                v[c + 1] = ex2(v[c + 1]);
            }
            if (!(ok = warp_wait(&bar.dpfull[buf], Cols::kDp == 2 ? (j >> 1) & 1 : j & 1, a.err,
                                 ERR_TIMEOUT_EPILOGUE)))
                break;
            tc_fence_after();
            const uint32_t tDP = tmem + lofs + Cols::DP + buf * kTile + half * 64;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float g[32];
                tmem_ld32(tDP + 32 * q, g);
                tmem_wait_ld();
                tmem_reg_fence(g);
#pragma unroll
                for (int c = 0; c < 32; ++c) v[32 * q + c] *= g[c] - delta;
            }
            if (!all_count(w)) {
                const uint32_t lo = half ? w.z : w.x, hi = half ? w.w : w.y;
#pragma unroll
                for (int c = 0; c < 64; ++c)
                    if (!(((c < 32 ? lo : hi) >> (c & 31)) & 1u)) v[c] = 0.f;
            }
            {
                uint32_t u[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) u[c] = pack16<BF>(v[2 * c], v[2 * c + 1]);
                tmem_st32(tDP, u);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.dsfull);
            }
            if (a.bias_part) {
                if (where != 0) {
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int c = 0; c < 64; c += 2) {
                        s0 += v[c];
                        s1 += v[c + 1];
                    }
                    if (where > 0)
                        far_hi += s0 + s1;
                    else
                        far_lo += s0 + s1;
                } else {
                    // sums along the diagonals: each lane's running sum moves one row down
                    // per column; lane 31's is complete.  A diagonal of these 32 rows meets
                    // two 64-column strips at most, so no entry gets more than two terms and
                    // the order of the additions does not matter.
                    float* sums = sSums + quarter * width;
                    auto put = [&](int64_t rel, float x) {
                        if (rel >= a.D)
                            far_hi += x;
                        else if (rel <= -a.D)
                            far_lo += x;
                        else
                            atomicAdd(sums + (int)rel + a.D, x);
                    };
                    float run = 0.f;
#pragma unroll
                    for (int c = 0; c < 64; ++c) {
                        run = __shfl_up_sync(0xffffffffu, run, 1);
                        run = (lane == 0 ? 0.f : run) + v[c];
                        if (lane == 31) put(rel0 + c - 31, run);
                        __syncwarp();
                    }
                    if (lane != 31) put(rel0 + 63 - lane, run);
                    __syncwarp();
                }
            }
        }
        if (nt > 0 && ok) ok = warp_wait(&bar.done, 0, a.err, ERR_TIMEOUT_EPILOGUE);
        if (ok) {
            tc_fence_after();
            const int mid = (dsteps * 16 + 31) / 32 * 16;
            store_row<BF>(a.dq, b * a.dq.sb + (int64_t)i * a.dq.st + h * a.dq.sh, tmem + lofs + Cols::DQ,
                          half ? mid : 0, half ? dsteps * 16 : mid, a.d, a.scale, nt > 0, live, true,
                          P.dq_vec);
        }
        if (a.bias_part) {
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                far_lo += __shfl_xor_sync(0xffffffffu, far_lo, o);
                far_hi += __shfl_xor_sync(0xffffffffu, far_hi, o);
            }
            if (lane == 0) {
                sFar[2 * warp] = far_lo;
                sFar[2 * warp + 1] = far_hi;
            }
            named_sync(1, 32 * kElemWarps);
            float* out = a.bias_part + ((int64_t)h * a.B * P.q_tiles + (int64_t)b * P.q_tiles + qt) * width;
            for (int e = threadIdx.x; e < width; e += 32 * kElemWarps) {
                float s = 0.f;
                if (e == 0 || e == width - 1) {
#pragma unroll
                    for (int k = 0; k < kElemWarps; ++k) s += sFar[2 * k + (e ? 1 : 0)];
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) s += sSums[k * width + e];
                }
                out[e] = s;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------

template <int HD, bool BF>
__global__ void __launch_bounds__(kGradThreads, 1) k_grad_kv(const __grid_constant__ GradArgs P) {
    constexpr uint32_t cS = 0, cDP = kTile, cDV = 2 * kTile, cDK = 3 * kTile;
    constexpr int kChunks = HD / 64, kTileBytes = kChunks * CHUNK_BYTES;
    constexpr uint64_t kTileU = kTileBytes >> 4;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    const Args& a = P.a;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int NS = P.kv_stages;           // even: Q and dO tiles in turn
    uint8_t* sK = smem;
    uint8_t* sV = sK + kTileBytes;
    uint8_t* sR = sV + kTileBytes;
    float* sRow = reinterpret_cast<float*>(sR + NS * kTileBytes);   // [NS / 2][-lse2 128, delta 128]
    GradBars& bar = *reinterpret_cast<GradBars*>(sRow + (NS / 2) * 2 * kTile);
    float* sBias = reinterpret_cast<float*>(&bar + 1);

    int blk = blockIdx.x;
    const int kt = blk % P.k_tiles;
    blk /= P.k_tiles;
    const int g = blk % a.G;
    const int b = blk / a.G;
    const int j0 = kt * kTile;
    const int end = key_end(a, b);
    uint4 w = make_uint4(0, 0, 0, 0);
    if (j0 < end) w = tile_words(P.kt, b, kt, end);
    const bool any = (w.x | w.y | w.z | w.w) != 0;
    const int64_t pos = a.q_pos ? (int64_t)__ldg(a.q_pos + b) : 0;
    const int dsteps = (a.d + 15) >> 4;
    const int nt = any ? a.R * P.q_tiles : 0;       // query tiles of every head

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&bar.full[s], 1);
            mbar_init(&bar.empty[s], 1);
        }
        mbar_init(&bar.ready, 1);
        mbar_init(&bar.sfull, 1);
        mbar_init(&bar.dpfull[0], 1);
        mbar_init(&bar.pfull, kElemWarps);
        mbar_init(&bar.dsfull, kElemWarps);
        mbar_init(&bar.done, 1);
        mbar_init(&bar.drain, 1);
        fence_mbar_init();
    }
    if (warp == 9) tmem_alloc(&bar.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;

    if (warp == 8) {
        if (nt > 0 && elect_one()) {
            mbar_arrive_expect_tx(&bar.ready, 2 * kTileBytes);
            for (int c = 0; c < kChunks; ++c) {
                tma_load(sK + c * CHUNK_BYTES, &P.k.map, c * 64, j0, g * P.k.head, b * P.k.batch, &bar.ready);
                tma_load(sV + c * CHUNK_BYTES, &P.v.map, c * 64, j0, g * P.v.head, b * P.v.batch, &bar.ready);
            }
            Ring r;
            int issued = 0;
            bool ok = true;
            int h = g * a.R, qt = 0;
            for (int it = 0; it < 2 * nt; ++it) {
                if (!mbar_wait(&bar.empty[r.slot], r.phase ^ 1u, a.err, ERR_TIMEOUT_PRODUCER)) {
                    ok = false;
                    break;
                }
                const bool second = it & 1;
                const TensorMap& src = second ? P.dout : P.q;
                // the row values come with Q: -lse2 and delta of the tile's queries
                mbar_arrive_expect_tx(&bar.full[r.slot], kTileBytes + (second ? 0 : 8 * kTile));
                for (int c = 0; c < kChunks; ++c)
                    tma_load(sR + r.slot * kTileBytes + c * CHUNK_BYTES, &src.map, c * 64, qt * kTile,
                             h * src.head, b * src.batch, &bar.full[r.slot]);
                if (!second)
                    bulk_g2s(sRow + (r.slot >> 1) * 2 * kTile,
                             P.rows + (((int64_t)b * a.H + h) * P.q_tiles + qt) * 2 * kTile, 8 * kTile,
                             &bar.full[r.slot]);
                ++issued;
                r.step(1, NS);
                if (second && ++qt == P.q_tiles) {
                    qt = 0;
                    ++h;
                }
            }
            if (!ok) {
                mbar_wait(&bar.ready, 0, a.err, ERR_TIMEOUT_PRODUCER);
                Ring l;
                for (int it = 0; it < issued; ++it) {
                    if (it + NS >= issued)
                        mbar_wait(&bar.full[l.slot], l.phase, a.err, ERR_TIMEOUT_PRODUCER);
                    l.step(1, NS);
                }
            }
        }
    } else if (warp == 9) {
        if (nt > 0 && elect_one()) {
            const uint32_t idS = idesc_16(BF, kTile, false);
            const uint32_t idD = idesc_16(BF, dsteps * 16, true);
            const uint64_t dK = sdesc_sw128(smem_u32(sK)), dV = sdesc_sw128(smem_u32(sV));
            const uint64_t dR = sdesc_sw128(smem_u32(sR)), dRt = sdesc_tokens(smem_u32(sR));
            Ring rs;               // the tile whose scores come next: Q at slot, dO at slot + 1
            Ring rd;               // the tile whose dV and dK come next
            bool ok = mma_wait(a.err, &bar.ready, 0) && mma_wait(a.err, &bar.full[0], 0);
            if (ok) {
                mma_over_d(tmem + cS, dK, dR, idS, dsteps);
                mma_commit(&bar.sfull);
                ok = mma_wait(a.err, &bar.full[1], 0);
            }
            if (ok) {
                mma_over_d(tmem + cDP, dV, dR + kTileU, idS, dsteps);
                mma_commit(&bar.dpfull[0]);
                rs.step(2, NS);
            }
            for (int t = 0; t < nt && ok; ++t) {
                const bool more = t + 1 < nt;
                if (!(ok = mma_wait(a.err, &bar.pfull, t & 1))) break;
                mma_over_tokens(tmem + cDV, tmem + cS, dRt + (rd.slot + 1) * kTileU, idD, t > 0, 64);
                mma_commit(&bar.empty[rd.slot + 1]);
                if (more) {
                    if (!(ok = mma_wait(a.err, &bar.full[rs.slot], rs.phase))) break;
                    mma_over_d(tmem + cS, dK, dR + rs.slot * kTileU, idS, dsteps);
                    mma_commit(&bar.sfull);
                }
                if (!(ok = mma_wait(a.err, &bar.dsfull, t & 1))) break;
                mma_over_tokens(tmem + cDK, tmem + cDP, dRt + rd.slot * kTileU, idD, t > 0, 64);
                mma_commit(&bar.empty[rd.slot]);
                rd.step(2, NS);
                if (more) {
                    if (!(ok = mma_wait(a.err, &bar.full[rs.slot + 1], rs.phase))) break;
                    mma_over_d(tmem + cDP, dV, dR + (rs.slot + 1) * kTileU, idS, dsteps);
                    mma_commit(&bar.dpfull[0]);
                    rs.step(2, NS);
                }
            }
            mma_commit(&bar.done);
            mma_commit(&bar.drain);
            mbar_wait(&bar.drain, 0, a.err, ERR_TIMEOUT_MMA);
        }
    } else if (warp < kElemWarps) {
        const int quarter = warp & 3, half = warp >> 2;
        const int r = quarter * 32 + lane;
        const int j = j0 + r;
        const uint32_t lofs = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + lofs + cS + half * 64, tDP = tmem + lofs + cDP + half * 64;
        Ring ring;
        bool ok = true;
        int h = g * a.R, qt = 0;
        for (int t = 0; t < nt; ++t) {
            if (a.table && qt == 0) {
                named_sync(1, 32 * kElemWarps);
                fill_bias<BF>(a, h, sBias, threadIdx.x, 32 * kElemWarps);
                named_sync(1, 32 * kElemWarps);
            }
            // relative position of the tile's first key and the strip's first query
            const int64_t rel0 = (int64_t)j0 - pos - (int64_t)qt * kTile - half * 64;
            const float* rows = sRow + (ring.slot >> 1) * 2 * kTile + half * 64;
            // (a warp that gave up still meets the others at the barriers above)
            ok = ok && warp_wait(&bar.full[ring.slot], ring.phase, a.err, ERR_TIMEOUT_EPILOGUE) &&
                 warp_wait(&bar.sfull, t & 1, a.err, ERR_TIMEOUT_EPILOGUE);
            if (ok) {
                tc_fence_after();
                float v[64];
                tmem_ld32(tS, v);
                tmem_ld32(tS + 32, v + 32);
                tmem_wait_ld();
                tmem_reg_fence(v);
                float mul = a.scale2, add = 0.f;
                if (a.table) {
                    if (rel0 - 63 >= a.D) {
                        add = sBias[2 * a.D + kSlack];
                    } else if (rel0 + (kTile - 1) <= -a.D) {
                        add = sBias[kSlack];
                    } else {
                        const float* e = sBias + (int)rel0 + r + a.D + kSlack;
#pragma unroll
                        for (int c = 0; c < 64; ++c) v[c] = fmaf(v[c], mul, e[-c]);
                        mul = 1.f;
                    }
                }
                const uint64_t mul2 = pk(mul, mul), add2_ = pk(add, add);
#pragma unroll
                for (int c = 0; c < 64; c += 4) {
                    const float4 l = *reinterpret_cast<const float4*>(rows + c);
                    upk(fma2(pk(v[c], v[c + 1]), mul2, add2(pk(l.x, l.y), add2_)), v[c], v[c + 1]);
                    upk(fma2(pk(v[c + 2], v[c + 3]), mul2, add2(pk(l.z, l.w), add2_)), v[c + 2], v[c + 3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[c + e] = ex2(v[c + e]);
                }
                {
                    uint32_t u[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) u[c] = pack16<BF>(v[2 * c], v[2 * c + 1]);
                    tmem_st32(tS, u);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.pfull);
                }
                ok = warp_wait(&bar.dpfull[0], t & 1, a.err, ERR_TIMEOUT_EPILOGUE);
                if (ok) {
                    tc_fence_after();
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float d[32];
                        tmem_ld32(tDP + 32 * q, d);
                        tmem_wait_ld();
                        tmem_reg_fence(d);
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 l = *reinterpret_cast<const float4*>(rows + kTile + 32 * q + c);
                            v[32 * q + c] *= d[c] - l.x;
                            v[32 * q + c + 1] *= d[c + 1] - l.y;
                            v[32 * q + c + 2] *= d[c + 2] - l.z;
                            v[32 * q + c + 3] *= d[c + 3] - l.w;
                        }
                    }
                    {
                        uint32_t u[32];
#pragma unroll
                        for (int c = 0; c < 32; ++c) u[c] = pack16<BF>(v[2 * c], v[2 * c + 1]);
                        tmem_st32(tDP, u);
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.dsfull);
                    }
                }
            }
            ring.step(2, NS);
            if (++qt == P.q_tiles) {
                qt = 0;
                ++h;
            }
        }
        if (nt > 0 && ok) ok = warp_wait(&bar.done, 0, a.err, ERR_TIMEOUT_EPILOGUE);
        if (ok) {
            tc_fence_after();
            const uint32_t word = quarter == 0 ? w.x : quarter == 1 ? w.y : quarter == 2 ? w.z : w.w;
            const bool keep = (word >> lane) & 1u;
            const bool live = j < a.m;
            const int mid = (dsteps * 16 + 31) / 32 * 16;
            const int c0 = half ? mid : 0, c1 = half ? dsteps * 16 : mid;
            store_row<BF>(a.dv, b * a.dv.sb + (int64_t)j * a.dv.st + g * a.dv.sh, tmem + lofs + cDV, c0, c1,
                          a.d, 1.f, nt > 0, live, keep, P.dv_vec);
            store_row<BF>(a.dk, b * a.dk.sb + (int64_t)j * a.dk.st + g * a.dk.sh, tmem + lofs + cDK, c0, c1,
                          a.d, a.scale, nt > 0, live, keep, P.dk_vec);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// dbias of one row of the table: the blocks' sums by relative position, in
// their order, then the positions of each bucket in theirs.

constexpr int kBiasThreads = 512;

template <bool BF>
__global__ void __launch_bounds__(kBiasThreads) k_grad_bias(const __grid_constant__ GradArgs P,
                                                            Elem<BF>* __restrict__ dbias) {
    extern __shared__ float sSum[];
    const Args& a = P.a;
    const int width = 2 * a.D + 1;
    const int64_t parts = (int64_t)a.B * P.q_tiles * (a.table_stride ? 1 : a.H);
    const float* src = a.bias_part + blockIdx.x * parts * width;
    for (int e = threadIdx.x; e < width; e += kBiasThreads) {
        float s = 0.f;
        for (int64_t p = 0; p < parts; ++p) s += src[p * width + e];
        sSum[e] = s;
    }
    __syncthreads();
    for (int u = threadIdx.x; u < a.nb; u += kBiasThreads) {
        float s = 0.f;
        for (int e = 0; e < width; ++e)
            if (bucket_of(a, e - a.D) == u) s += sSum[e];
        dbias[(int64_t)blockIdx.x * a.nb + u] = from_f<Elem<BF>>(s);
    }
}

// ---------------------------------------------------------------------------

int ring_stages(size_t fixed, size_t per_stage) {
    const int s = (int)((kSmemLimit - fixed) / per_stage);
    return s < kMaxRing ? s : kMaxRing;
}

template <int HD, bool BF>
cudaError_t launch_grad(GradArgs p, void* dbias, cudaStream_t s) {
    const Args& a = p.a;
    constexpr size_t tile = (HD / 64) * CHUNK_BYTES;
    const size_t bias = a.table ? sizeof(float) * (2 * (size_t)(a.D + kSlack) + 1) : 0;
    const size_t width = 2 * (size_t)a.D + 1;
    static std::atomic<uint64_t> ready_q{0}, ready_kv{0};
    cudaError_t e;
    if (a.n > 0) {
        const size_t fixed = 1024 + sizeof(GradBars) + sizeof(float) * (kTile + 2 * kElemWarps) + bias +
                             (a.bias_part ? sizeof(float) * kBands * width : 0);
        p.stages = 2 * (ring_stages(fixed, tile) / 2);     // even: K keeps its slots, and their clean bars
        if ((e = raise_smem(k_grad_q<HD, BF>, kSmemLimit, ready_q)) != cudaSuccess) return e;
        k_grad_q<HD, BF><<<(unsigned)((int64_t)p.q_tiles * a.H * a.B), kGradThreads,
                           fixed + p.stages * tile, s>>>(p);
        count_launch();
    }
    if (a.m > 0) {
        // K and V, then stages of which each pair has a row of (-lse2, delta)
        const size_t fixed = 1024 + sizeof(GradBars) + bias + 2 * tile;
        p.kv_stages = 2 * (ring_stages(fixed, tile + 4 * kTile) / 2);
        if ((e = raise_smem(k_grad_kv<HD, BF>, kSmemLimit, ready_kv)) != cudaSuccess) return e;
        k_grad_kv<HD, BF><<<(unsigned)((int64_t)p.k_tiles * a.G * a.B), kGradThreads,
                            fixed + p.kv_stages * (tile + 4 * kTile), s>>>(p);
        count_launch();
    }
    if (dbias) {
        k_grad_bias<BF><<<a.table_stride ? a.H : 1, kBiasThreads, sizeof(float) * width, s>>>(
            p, static_cast<Elem<BF>*>(dbias));
        count_launch();
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_grad_tc(const GradArgs& p, void* dbias, cudaStream_t s) {
    if (p.a.d <= 64) return p.a.bf16 ? launch_grad<64, true>(p, dbias, s) : launch_grad<64, false>(p, dbias, s);
    return p.a.bf16 ? launch_grad<128, true>(p, dbias, s) : launch_grad<128, false>(p, dbias, s);
}

}  // namespace attn
}  // namespace fs
