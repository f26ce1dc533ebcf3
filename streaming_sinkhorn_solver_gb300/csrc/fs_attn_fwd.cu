// Cross attention, forward, on the tensor cores.
//
// A block takes 256 queries of one head in two tiles of 128 and streams the
// keys in tiles of 128:
//   S_t = Q_t K^T (TMEM), p = 2^{x - ref} in 16 bits over S_t in TMEM,
//   O_t += P_t V (TMEM, P as the A operand read from TMEM).
// One warp issues the copies, one thread the products, four warps per query
// tile hold a row per thread and keep its running sum and reference.  While
// one tile's rows are in the softmax, the tensor core works on the other's
// products; V is read as an operand summed over its rows, so nothing is
// transposed.
//
// The reference is the running maximum, moved only when a row's maximum grew
// by more than 2^8 (p then stays below 256, which both types and the float32
// sums hold with the same relative precision); the rare move rescales O_t in
// TMEM.
#include "fs_attn_host.cuh"

#include <atomic>
#include <type_traits>

namespace fs {
namespace attn {

namespace {

constexpr int kFwdThreads = 384;
constexpr int kSlack = 2 * kTile;          // bias table entries beyond +-D on each side
constexpr float kRefSlack = 8.f;

template <int HD>
struct Fwd {
    static constexpr int kChunks = HD / 64;
    static constexpr int kTileBytes = kChunks * CHUNK_BYTES;
    static constexpr int kStages = HD == 64 ? 6 : 4;   // K and V tiles in turn
    static constexpr int kBars = 1 + 3 * kStages + 2 + 2 + 1 + 1;
    static constexpr size_t kFixed = 1024 + (size_t)(2 + kStages) * kTileBytes + 8 * kBars + 16;
};

// One row's result from its sum and O in TMEM: out and lse, or the partial of
// this split.  Whole warps.
template <bool BF>
__device__ __forceinline__ void write_row(const FwdArgs& P, uint32_t tO, int b, int h, int i, int split,
                                          bool any, int dsteps, float ref, float sum) {
    using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    const Args& a = P.a;
    const bool live = i < a.n;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const float lse2 = sum == 0.f ? -INFINITY : ref + lg2(sum);
    const int64_t row = ((int64_t)b * a.H + h) * a.n + i;
    float* part = P.splits > 1 ? P.part.out + (split * P.part.rows + row) * a.d : nullptr;
    T* out = static_cast<T*>(a.o.p) + b * a.o.sb + (int64_t)i * a.o.st + h * a.o.sh;
    for (int c = 0; c < dsteps * 16; c += 16) {
        float o[16];
        if (any) {
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
        } else if (P.out_vec) {
#pragma unroll
            for (int e = 0; e < 16; e += 8)
                if (live && c + e < a.d)
                    *reinterpret_cast<uint4*>(out + c + e) =
                        make_uint4(pack16<BF>(o[e], o[e + 1]), pack16<BF>(o[e + 2], o[e + 3]),
                                   pack16<BF>(o[e + 4], o[e + 5]), pack16<BF>(o[e + 6], o[e + 7]));
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (live && c + e < a.d) out[c + e] = from_f<T>(o[e]);
        }
        __syncwarp();
    }
    if (!live) return;
    if (part)
        P.part.lse2[split * P.part.rows + row] = lse2;
    else
        a.lse[row] = lse2 * (float)kLn2;
}

template <int HD, bool BF>
__global__ void __launch_bounds__(kFwdThreads, 1) k_forward_tc(const __grid_constant__ FwdArgs P) {
    using C = Fwd<HD>;
    constexpr int NS = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    const Args& a = P.a;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    uint8_t* sQ = smem;
    uint8_t* sKV = sQ + 2 * C::kTileBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(sKV + NS * C::kTileBytes);
    uint64_t* empty = full + NS;
    uint64_t* clean = empty + NS;     // a V tile whose uncounted rows are zero
    uint64_t* qfull = clean + NS;
    uint64_t* sfull = qfull + 1;
    uint64_t* pfull = sfull + 2;
    uint64_t* ofull = pfull + 2;
    uint64_t* drain = ofull + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    float* sBias = reinterpret_cast<float*>(tmem_slot + 4);

    int blk = blockIdx.x;
    const int split = blk % P.splits;
    blk /= P.splits;
    const int qt = blk % P.row_blocks;
    blk /= P.row_blocks;
    const int h = blk % a.H;
    const int b = blk / a.H;
    const int i0 = qt * 2 * kTile;
    const bool two = i0 + kTile < a.n;
    const int end = key_end(a, b);
    const int nt_all = tile_count(P.kt, b, end);
    const int per = (nt_all + P.splits - 1) / P.splits;
    const int t0 = min(nt_all, split * per);
    const int nt = min(nt_all, t0 + per) - t0;
    const bool partial_keys = P.kt.words != nullptr || end < a.m;
    const int64_t pos = a.q_pos ? (int64_t)__ldg(a.q_pos + b) : 0;
    const int dsteps = (a.d + 15) >> 4;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&clean[s], 1);
        }
        mbar_init(qfull, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sfull[t], 1);
            mbar_init(&pfull[t], 4);
        }
        mbar_init(ofull, 1);
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    if (warp == 9) tmem_alloc(tmem_slot, 512);
    if (a.table) {
        // base-2 bias by relative position -D - kSlack .. D + kSlack of this head
        using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
        const T* row = static_cast<const T*>(a.table) + h * a.table_stride;
        for (int e = threadIdx.x; e < 2 * (a.D + kSlack) + 1; e += kFwdThreads)
            sBias[e] = bias2(to_f<T>(row[bucket_of(a, (int64_t)e - a.D - kSlack)]));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 8) {
        if (nt > 0 && elect_one()) {
            const int g = h / a.R;
            mbar_arrive_expect_tx(qfull, (two ? 2 : 1) * C::kTileBytes);
            for (int t = 0; t < (two ? 2 : 1); ++t)
                for (int c = 0; c < C::kChunks; ++c)
                    tma_load(sQ + t * C::kTileBytes + c * CHUNK_BYTES, &P.q.map, c * 64, i0 + t * kTile,
                             h * P.q.head, b * P.q.batch, qfull);
            int issued = 0;
            bool ok = true;
            for (int it = 0; it < 2 * nt; ++it) {
                const int s = it % NS;
                if (!mbar_wait(&empty[s], ((it / NS) & 1) ^ 1, a.err, ERR_TIMEOUT_PRODUCER)) {
                    ok = false;
                    break;
                }
                const int tile = tile_at(P.kt, b, t0 + (it >> 1));
                const TensorMap& src = it & 1 ? P.v : P.k;
                mbar_arrive_expect_tx(&full[s], C::kTileBytes);
                for (int c = 0; c < C::kChunks; ++c)
                    tma_load(sKV + s * C::kTileBytes + c * CHUNK_BYTES, &src.map, c * 64, tile * kTile,
                             g * src.head, b * src.batch, &full[s]);
                ++issued;
            }
            if (!ok) {   // every copy lands before the block can exit
                mbar_wait(qfull, 0, a.err, ERR_TIMEOUT_PRODUCER);
                for (int it = max(0, issued - NS); it < issued; ++it)
                    mbar_wait(&full[it % NS], (it / NS) & 1, a.err, ERR_TIMEOUT_PRODUCER);
            }
        }
    } else if (warp == 9) {
        if (nt > 0 && elect_one()) {
            const uint32_t idS = idesc_16(BF, kTile, false);
            const uint32_t idO = idesc_16(BF, dsteps * 16, true);
            const uint64_t dQ = sdesc_sw128(smem_u32(sQ)), dK = sdesc_sw128(smem_u32(sKV));
            const uint64_t dV = sdesc_tokens(smem_u32(sKV));
            constexpr uint64_t kTileU = C::kTileBytes >> 4;    // descriptors count 16 bytes
            bool ok = mbar_wait(qfull, 0, a.err, ERR_TIMEOUT_MMA) &&
                      mbar_wait(&full[0], 0, a.err, ERR_TIMEOUT_MMA);
            if (ok) {
                tc_fence_after();
                mma_over_d(tmem, dQ, dK, idS, dsteps);
                mma_commit(&sfull[0]);
                if (two) {
                    mma_over_d(tmem + kTile, dQ + kTileU, dK, idS, dsteps);
                    mma_commit(&sfull[1]);
                }
                mma_commit(&empty[0]);
            }
            for (int j = 0; j < nt && ok; ++j) {
                const int vs = (2 * j + 1) % NS, ks = (2 * j + 2) % NS;
                if (!mbar_wait(partial_keys ? &clean[vs] : &full[vs], ((2 * j + 1) / NS) & 1, a.err,
                               ERR_TIMEOUT_MMA)) {
                    ok = false;
                    break;
                }
                const bool more = j + 1 < nt;
                if (more && !mbar_wait(&full[ks], ((2 * j + 2) / NS) & 1, a.err, ERR_TIMEOUT_MMA)) {
                    ok = false;
                    break;
                }
                for (int t = 0; t < (two ? 2 : 1); ++t) {
                    if (!mbar_wait(&pfull[t], j & 1, a.err, ERR_TIMEOUT_MMA)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    mma_over_tokens(tmem + (2 + t) * kTile, tmem + t * kTile, dV + vs * kTileU, idO, j > 0);
                    if (more) {
                        mma_over_d(tmem + t * kTile, dQ + t * kTileU, dK + ks * kTileU, idS, dsteps);
                        mma_commit(&sfull[t]);
                    }
                }
                if (!ok) break;
                mma_commit(&empty[vs]);
                if (more) mma_commit(&empty[ks]);
            }
            mma_commit(ofull);
            mma_commit(drain);
            mbar_wait(drain, 0, a.err, ERR_TIMEOUT_MMA);
        }
    } else if (warp == 10) {
        if (partial_keys) {
            for (int j = 0; j < nt; ++j) {
                const int vs = (2 * j + 1) % NS;
                const uint4 w = tile_words(P.kt, b, tile_at(P.kt, b, t0 + j), end);
                if (!warp_wait(&full[vs], ((2 * j + 1) / NS) & 1, a.err, ERR_TIMEOUT_PRODUCER)) break;
                if (!all_count(w)) {
                    clear_rows(sKV + vs * C::kTileBytes, C::kChunks, w, lane);
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&clean[vs]);
            }
        }
    } else if (warp < 8) {
        const int t = warp >> 2;
        if (t == 0 || two) {
            const int r = (warp & 3) * 32 + lane;
            const int i = i0 + t * kTile + r;
            const uint32_t lofs = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t tS = tmem + t * kTile + lofs, tO = tmem + (2 + t) * kTile + lofs;
            const int64_t first = pos + i0 + t * kTile;          // position of the tile's first query
            float ref = -INFINITY, sum = 0.f;
            bool ok = true;
            for (int j = 0; j < nt; ++j) {
                const int tile = tile_at(P.kt, b, t0 + j);
                const uint4 w = tile_words(P.kt, b, tile, end);
                const int64_t rel0 = (int64_t)tile * kTile - first;   // of the tile's first row and key
                if (!warp_wait(&sfull[t], j & 1, a.err, ERR_TIMEOUT_EPILOGUE)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                float v[kTile];
#pragma unroll
                for (int c = 0; c < kTile; c += 32) tmem_ld32(tS + c, v + c);
                tmem_wait_ld();
                tmem_reg_fence(v);
                float mul = a.scale2, add = 0.f;
                if (a.table) {
                    if (rel0 - (kTile - 1) >= a.D) {
                        add = sBias[2 * a.D + kSlack];
                    } else if (rel0 + (kTile - 1) <= -a.D) {
                        add = sBias[kSlack];
                    } else {
                        // |rel| < D + 2 * 128 here
                        const float* e = sBias + (int)rel0 - r + a.D + kSlack;
#pragma unroll
                        for (int c = 0; c < kTile; ++c) v[c] = fmaf(v[c], mul, e[c]);
                        mul = 1.f;
                    }
                }
                if (!all_count(w)) {
                    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int c = 0; c < kTile; ++c)
                        if (!((words[c >> 5] >> (c & 31)) & 1u)) v[c] = -INFINITY;
                }
                float m0 = v[0], m1 = v[1], m2 = v[2], m3 = v[3];
#pragma unroll
                for (int c = 4; c < kTile - 4; c += 8) {
                    m0 = max3(m0, v[c], v[c + 1]);
                    m1 = max3(m1, v[c + 2], v[c + 3]);
                    m2 = max3(m2, v[c + 4], v[c + 5]);
                    m3 = max3(m3, v[c + 6], v[c + 7]);
                }
                m0 = max3(m0, v[kTile - 4], v[kTile - 3]);
                m1 = max3(m1, v[kTile - 2], v[kTile - 1]);
                const float top = fmaf(fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)), mul, add);
                float alpha = 1.f;
                if (top > ref + kRefSlack) {
                    // (up to its first counted key a row's sum and O are zero)
                    if (ref != -INFINITY) alpha = ex2(ref - top);
                    sum *= alpha;
                    ref = top;
                }
                if (__any_sync(0xffffffffu, alpha != 1.f)) {
                    // the products of tile j - 1 are complete: S of tile j came after them
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
                const float base = add - (ref == -INFINITY ? 0.f : ref);
                const uint64_t mul2 = pk(mul, mul), base2 = pk(base, base);
                uint64_t s0 = 0, s1 = 0;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t p[32];
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const int x = half * 64 + 2 * c;
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
                    tmem_st32(tS + half * 32, p);
                }
                float a0, a1, b0, b1;
                upk(s0, a0, a1);
                upk(s1, b0, b1);
                sum += (a0 + a1) + (b0 + b1);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[t]);
            }
            if (nt > 0 && ok) ok = warp_wait(ofull, 0, a.err, ERR_TIMEOUT_EPILOGUE);
            if (ok) {
                tc_fence_after();
                write_row<BF>(P, tO, b, h, i, split, nt > 0, dsteps, ref, sum);
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

template <int HD, bool BF>
cudaError_t launch_forward(const FwdArgs& p, cudaStream_t s) {
    const size_t bias = p.a.table ? sizeof(float) * (2 * (size_t)(p.a.D + kSlack) + 1) : 0;
    constexpr size_t most = Fwd<HD>::kFixed + sizeof(float) * (2 * (size_t)(kMaxDistance + kSlack) + 1);
    static_assert(most <= kSmemLimit, "forward kernel does not fit in shared memory");
    static std::atomic<uint64_t> ready{0};    // devices whose shared-memory limit is raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!(ready.load() >> dev & 1)) {
        e = cudaFuncSetAttribute(k_forward_tc<HD, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)most);
        if (e != cudaSuccess) return e;
        ready.fetch_or(1ull << dev);
    }
    const unsigned blocks = (unsigned)((int64_t)p.row_blocks * p.a.H * p.a.B * p.splits);
    k_forward_tc<HD, BF><<<blocks, kFwdThreads, Fwd<HD>::kFixed + bias, s>>>(p);
    count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_forward_tc(const FwdArgs& p, cudaStream_t s) {
    if (p.a.d <= 64)
        return p.a.bf16 ? launch_forward<64, true>(p, s) : launch_forward<64, false>(p, s);
    return p.a.bf16 ? launch_forward<128, true>(p, s) : launch_forward<128, false>(p, s);
}

}  // namespace attn
}  // namespace fs
