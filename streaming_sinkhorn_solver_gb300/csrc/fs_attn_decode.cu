// Cross attention of few queries against many keys (single tokens against a
// cache): bound by reading the keys and values once.
//
// The R n query rows that share a key head are one tile of 8 or 16 rows, so a
// key is read once for all of them.  Blocks split the keys of a (batch, key
// head); a warp takes 16 or 32 keys at a time straight from memory into the operand
// registers of mma.sync (the tensor core's 128-row tiles would be empty here,
// and nothing needs shared memory):
//   S (rows x keys) = Q K^T: the 16 elements of a product may be any 16 of the
//     d, the same for both operands, so a lane's 16-byte piece of a key row is
//     two products' worth of its operand as it comes;
//   O^T (d x rows) += V^T P^T: a lane holds the same 16 bytes of four value
//     rows, and four byte permutes make each operand of two d of it; P^T is S's
//     own register layout.
// Softmax as in the forward kernel (float32, a reference that moves only past
// 2^8).  In bfloat16 P is split into two parts of 8 bits each, so its rounding
// does not show; the products are idle anyway.  In float16 it is one part of 11 bits
// (out 0.026 % off in the 2-norm, of which 0.021 % is its own rounding).  The warps' results are joined in
// shared memory, the blocks' by the last block of a (batch, key head) to finish,
// in the order of the splits.
//
// Measured: 64 sequences, 32 heads on 8 of 128, one token each against 4096 keys: 170 us,
// 6.3 TB/s (0.93 of the measured copy rate), 140 us with lengths from half of that on;
// 2 x 2 tokens of 16 heads on 4 of 64 against 200001 keys with a position bias: 77 us,
// 4.9 TB/s; one token of 16 heads of 64 against 1500 keys: 11.6 us, latency.
#include "fs_attn_host.cuh"

#include <type_traits>

namespace fs {
namespace attn {

namespace {

constexpr int kWarps = 4;
// blocks of 16 keys that a warp takes at a time
constexpr int key_blocks(int HD) { return HD == 64 ? 1 : 2; }
constexpr int kBiasFloats = 8192;      // most bias entries kept in shared memory

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

__device__ __forceinline__ uint4 ld16(const uint16_t* p, bool on) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (on)
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "l"(p));
    return x;
}
__device__ __forceinline__ uint32_t word(const uint4& x, int k) {
    return k == 0 ? x.x : k == 1 ? x.y : k == 2 ? x.z : x.w;
}

// RB: blocks of 8 query rows
template <int HD, int RB>
constexpr size_t kDecodeSmem = sizeof(float) * kWarps * 8 * RB * (HD + 2);

template <int HD, bool BF, int RB>
__global__ void __launch_bounds__(32 * kWarps) k_decode(const __grid_constant__ DecodeArgs P) {
    using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    constexpr int U = HD / 32, W = HD / 64, RP = (RB + 1) / 2, ROWS = 8 * RB;
    constexpr int KB = key_blocks(HD), KEYS = 16 * KB;
    extern __shared__ float smem[];
    float* sO = smem;                                   // [warp][row][HD]
    float* sRef = sO + kWarps * ROWS * HD;              // [warp][row]
    float* sSum = sRef + kWarps * ROWS;
    float* sBias = sSum + kWarps * ROWS;                // [R][2 D + 1], where it fits
    __shared__ int sLast;
    const Args& a = P.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;

    int blk = blockIdx.x;
    const int split = blk % P.splits;
    blk /= P.splits;
    const int group = blk % P.groups;
    blk /= P.groups;
    const int kh = blk % a.G;
    const int b = blk / a.G;
    const int nrows = min(ROWS, a.R * a.n - group * ROWS);
    const int end = key_end(a, b);
    // this split's keys, in whole steps of the block
    const int steps = (end + kDecodeKeys - 1) / kDecodeKeys;
    const int per = (steps + P.splits - 1) / P.splits;
    const int k0 = (int)min((int64_t)end, (int64_t)split * per * kDecodeKeys);
    const int k1 = (int)min((int64_t)end, k0 + (int64_t)per * kDecodeKeys);
    const int64_t pos = a.q_pos ? (int64_t)__ldg(a.q_pos + b) : 0;
    const uint8_t* mask = a.mask ? a.mask + (int64_t)b * a.mask_stride : nullptr;
    const int width = 2 * a.D + 1;

    // bias entries of this block's heads, if any pair of it is within +-D
    const bool near = a.table && k0 < k1 && k1 - 1 - pos > -a.D && k0 - pos - (a.n - 1) < a.D;
    const bool in_smem = near && a.R * width <= kBiasFloats;
    if (in_smem) {
        for (int e = threadIdx.x; e < a.R * width; e += 32 * kWarps) {
            const int r = e / width;
            const T* row = static_cast<const T*>(a.table) + (int64_t)(kh * a.R + r) * a.table_stride;
            sBias[e] = bias2(to_f<T>(row[bucket_of(a, (int64_t)(e - r * width) - a.D)]));
        }
        __syncthreads();
    }

    // Row 8 rb + g of the tile is query i = row % n of head kh R + row / n.
    uint4 q[RB][U];
    float lo[RB], hi[RB];                 // bias beyond -D and D
    int qi[RB], qr[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int row = group * ROWS + min(8 * rb + g, nrows - 1);
        qr[rb] = row / a.n;
        qi[rb] = row - qr[rb] * a.n;
        const uint16_t* p = static_cast<const uint16_t*>(a.q.p) + b * a.q.sb + qi[rb] * a.q.st +
                            (int64_t)(kh * a.R + qr[rb]) * a.q.sh;
#pragma unroll
        for (int u = 0; u < U; ++u) q[rb][u] = ld16(p + 8 * (t + 4 * u), 8 * (t + 4 * u) < a.d);
        lo[rb] = hi[rb] = 0.f;
        if (a.table) {
            const T* tr = static_cast<const T*>(a.table) + (int64_t)(kh * a.R + qr[rb]) * a.table_stride;
            lo[rb] = bias2(to_f<T>(tr[bucket_of(a, -a.D)]));
            hi[rb] = bias2(to_f<T>(tr[bucket_of(a, a.D)]));
        }
    }
    float ref[RB], sum[RB], o[RB][W][4][4];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        ref[rb] = -INFINITY;
        sum[rb] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[rb][w][r][e] = 0.f;
    }
    const uint16_t* kp = static_cast<const uint16_t*>(a.k.p) + b * a.k.sb + kh * a.k.sh + 8 * t;
    const uint16_t* vp = static_cast<const uint16_t*>(a.v.p) + b * a.v.sb + kh * a.v.sh + 8 * g;

    for (int key = k0 + KEYS * warp; key < k1; key += KEYS * kWarps) {
        // bits of the counted keys among these
        uint32_t bits = key + KEYS <= k1 ? (uint32_t)((1ull << KEYS) - 1) : (1u << (k1 - key)) - 1u;
        if (mask) {
            const bool on = ((bits >> lane) & 1u) && __ldg(mask + key + lane) != 0;
            bits = __ballot_sync(0xffffffffu, on);
            if (bits == 0) continue;
        }
        uint4 k[2 * KB][U], v[KB][4][W];
#pragma unroll
        for (int nb = 0; nb < 2 * KB; ++nb) {
            const int j = 8 * nb + g;
            const bool on = (bits >> j) & 1u;
            const uint16_t* p = kp + (int64_t)(key + j) * a.k.st;
#pragma unroll
            for (int u = 0; u < U; ++u) k[nb][u] = ld16(p + 32 * u, on && 8 * t + 32 * u < a.d);
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int j = 16 * kb + 2 * t + (x & 1) + 8 * (x >> 1);
                const bool on = (bits >> j) & 1u;
                const uint16_t* p = vp + (int64_t)(key + j) * a.v.st;
#pragma unroll
                for (int w = 0; w < W; ++w) v[kb][x][w] = ld16(p + 64 * w, on && 8 * g + 64 * w < a.d);
            }
        float s[RP][2 * KB][4];
#pragma unroll
        for (int rp = 0; rp < RP; ++rp)
#pragma unroll
            for (int nb = 0; nb < 2 * KB; ++nb) {
                float* c = s[rp][nb];
                c[0] = c[1] = c[2] = c[3] = 0.f;
                constexpr bool pair = RB > 1;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        mma16816<BF>(c, word(q[2 * rp][u], 2 * y),
                                     pair ? word(q[pair ? 2 * rp + 1 : 0][u], 2 * y) : 0u,
                                     word(q[2 * rp][u], 2 * y + 1),
                                     pair ? word(q[pair ? 2 * rp + 1 : 0][u], 2 * y + 1) : 0u,
                                     word(k[nb][u], 2 * y), word(k[nb][u], 2 * y + 1));
            }
        // scores of row 8 rb + g and keys 8 nb + 2 t + {0, 1}
        uint32_t ph[RB][2 * KB], pl[RB][2 * KB];
        float alpha[RB];
        bool moved = false;
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            float x[4 * KB], top = -INFINITY;
#pragma unroll
            for (int e = 0; e < 4 * KB; ++e) {
                const int j = 8 * (e >> 1) + 2 * t + (e & 1);
                float bias = 0.f;
                if (a.table) {
                    const int64_t rel = key + j - pos - qi[rb];
                    if (rel >= a.D)
                        bias = hi[rb];
                    else if (rel <= -a.D)
                        bias = lo[rb];
                    else if (in_smem)
                        bias = sBias[qr[rb] * width + (int)rel + a.D];
                    else
                        bias = bias2(to_f<T>(static_cast<const T*>(
                            a.table)[(int64_t)(kh * a.R + qr[rb]) * a.table_stride + bucket_of(a, rel)]));
                }
                x[e] = (bits >> j) & 1u ? fmaf(s[rb >> 1][e >> 1][2 * (rb & 1) + (e & 1)], a.scale2, bias)
                                        : -INFINITY;
                top = fmaxf(top, x[e]);
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            alpha[rb] = 1.f;
            if (top > ref[rb] + 8.f) {
                if (ref[rb] != -INFINITY) alpha[rb] = ex2(ref[rb] - top);
                sum[rb] *= alpha[rb];
                ref[rb] = top;
                moved |= alpha[rb] != 1.f;
            }
            const float base = (ref[rb] == -INFINITY ? 0.f : ref[rb]) - kProbShift<BF>;
#pragma unroll
            for (int e = 0; e < 4 * KB; ++e) {
                x[e] = ex2(x[e] - base);
                sum[rb] += x[e];
            }
#pragma unroll
            for (int nb = 0; nb < 2 * KB; ++nb) {
                const uint32_t h = pack16<BF>(x[2 * nb], x[2 * nb + 1]);
                ph[rb][nb] = h;
                if (BF)
                    pl[rb][nb] = pack16<BF>(x[2 * nb] - __uint_as_float(h << 16),
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
                for (int w = 0; w < W; ++w)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        o[rb][w][r][0] *= a0;
                        o[rb][w][r][1] *= a1;
                        o[rb][w][r][2] *= a0;
                        o[rb][w][r][3] *= a1;
                    }
            }
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int w = 0; w < W; ++w)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint4(&x)[4][W] = v[kb];
                    const uint32_t a0 = __byte_perm(word(x[0][w], r), word(x[1][w], r), 0x5410);
                    const uint32_t a1 = __byte_perm(word(x[0][w], r), word(x[1][w], r), 0x7632);
                    const uint32_t a2 = __byte_perm(word(x[2][w], r), word(x[3][w], r), 0x5410);
                    const uint32_t a3 = __byte_perm(word(x[2][w], r), word(x[3][w], r), 0x7632);
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb) {
                        mma16816<BF>(o[rb][w][r], a0, a1, a2, a3, ph[rb][2 * kb], ph[rb][2 * kb + 1]);
                        if (BF) mma16816<BF>(o[rb][w][r], a0, a1, a2, a3, pl[rb][2 * kb], pl[rb][2 * kb + 1]);
                    }
                }
    }

    // each warp's rows, then their join
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        sum[rb] += __shfl_xor_sync(0xffffffffu, sum[rb], 1);
        sum[rb] += __shfl_xor_sync(0xffffffffu, sum[rb], 2);
        if (t == 0) {
            sRef[warp * ROWS + 8 * rb + g] = ref[rb];
            sSum[warp * ROWS + 8 * rb + g] = sum[rb];
        }
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float* p = sO + (size_t)(warp * ROWS + 8 * rb + 2 * t) * HD + 8 * (g + 8 * w) + 2 * r;
                *reinterpret_cast<float2*>(p) = make_float2(o[rb][w][r][0], o[rb][w][r][2]);
                *reinterpret_cast<float2*>(p + HD) = make_float2(o[rb][w][r][1], o[rb][w][r][3]);
            }
    }
    __syncthreads();
    const int64_t head0 = (int64_t)b * a.H + kh * a.R;
    for (int row = warp; row < nrows; row += kWarps) {
        const int all = group * ROWS + row;
        const int r = all / a.n, i = all - r * a.n;
        const int64_t at = (head0 + r) * a.n + i;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sRef[w * ROWS + row]);
        const float base = top == -INFINITY ? 0.f : top;
        float total = 0.f, f[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            f[w] = ex2(sRef[w * ROWS + row] - base);
            total = fmaf(f[w], sSum[w * ROWS + row], total);
        }
        const float inv = total == 0.f ? 0.f : 1.f / total;
        const float lse2 = total == 0.f ? -INFINITY : top - kProbShift<BF> + lg2(total);
        T* out = static_cast<T*>(a.o.p) + b * a.o.sb + i * a.o.st + (int64_t)(kh * a.R + r) * a.o.sh;
        float* part = P.part.out + (split * P.part.rows + at) * P.dp;
        for (int c = lane; c < P.dp; c += 32) {
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) x = fmaf(f[w], sO[(size_t)(w * ROWS + row) * HD + c], x);
            x = total == 0.f ? 0.f : x * inv;
            if (P.splits > 1)
                part[c] = x;
            else if (c < a.d)
                out[c] = from_f<T>(x);
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
    static_assert(ROWS * kSome <= kWarps * ROWS * HD, "weights fit over the rows");
    float top[ROWS / kWarps], total[ROWS / kWarps];
#pragma unroll
    for (int x = 0; x < ROWS / kWarps; ++x) {
        const int row = warp + kWarps * x;
        top[x] = -INFINITY;
        total[x] = 0.f;
        if (row < nrows) {
            const float* l = P.part.lse2 + head0 * a.n + group * ROWS + row;   // rows (head, query)
            for (int s = lane; s < P.splits; s += 32) top[x] = fmaxf(top[x], l[s * P.part.rows]);
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
            const float* l = P.part.lse2 + head0 * a.n + group * ROWS + row;
            float sum = 0.f;
            for (int s = lane; s < some; s += 32) {
                const float w = ex2(l[(s0 + s) * P.part.rows] - (top[x] == -INFINITY ? 0.f : top[x]));
                sO[row * kSome + s] = w;
                sum += w;
            }
#pragma unroll
            for (int y = 16; y; y >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, y);
            total[x] += sum;
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kSums; ++x) {
            const int e = threadIdx.x + x * 32 * kWarps, row = e / kQuads, c = 4 * (e % kQuads);
            if (row >= nrows || c >= a.d) continue;
            const float* src = P.part.out + (s0 * P.part.rows + head0 * a.n + group * ROWS + row) * P.dp + c;
            const float* w = sO + row * kSome;
            const int64_t step = P.part.rows * P.dp;
#pragma unroll 16
            for (int s = 0; s < some; ++s) {
                const float4 y = *reinterpret_cast<const float4*>(src + s * step);
                acc[x].x = fmaf(w[s], y.x, acc[x].x);
                acc[x].y = fmaf(w[s], y.y, acc[x].y);
                acc[x].z = fmaf(w[s], y.z, acc[x].z);
                acc[x].w = fmaf(w[s], y.w, acc[x].w);
            }
        }
    }
#pragma unroll
    for (int x = 0; x < ROWS / kWarps; ++x) {
        const int row = warp + kWarps * x;
        if (lane == 0 && row < nrows) {
            sSum[row] = total[x];
            a.lse[head0 * a.n + group * ROWS + row] =
                total[x] == 0.f ? -INFINITY : (top[x] + lg2(total[x])) * (float)kLn2;
        }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kSums; ++x) {
        const int e = threadIdx.x + x * 32 * kWarps, row = e / kQuads, c = 4 * (e % kQuads);
        if (row >= nrows || c >= a.d) continue;
        const int all = group * ROWS + row;
        const int r = all / a.n, i = all - r * a.n;
        T* out = static_cast<T*>(a.o.p) + b * a.o.sb + i * a.o.st + (int64_t)(kh * a.R + r) * a.o.sh + c;
        const float inv = sSum[row] == 0.f ? 0.f : 1.f / sSum[row];
        const float y[4] = {acc[x].x * inv, acc[x].y * inv, acc[x].z * inv, acc[x].w * inv};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (c + k < a.d) out[k] = from_f<T>(y[k]);
    }
}

template <int HD, int RB>
size_t smem_bytes(const Args& a) {
    return kDecodeSmem<HD, RB> +
           (a.table ? sizeof(float) * (size_t)std::min(kBiasFloats, a.R * (2 * a.D + 1)) : 0);
}

template <int HD, bool BF, int RB>
cudaError_t launch(const DecodeArgs& p, cudaStream_t s) {
    constexpr size_t most = kDecodeSmem<HD, RB> + sizeof(float) * kBiasFloats;
    static std::atomic<uint64_t> ready{0};    // devices whose shared-memory limit is raised
    if (cudaError_t e = raise_smem(k_decode<HD, BF, RB>, most, ready); e != cudaSuccess) return e;
    const unsigned blocks = (unsigned)((int64_t)p.a.B * p.a.G * p.groups * p.splits);
    k_decode<HD, BF, RB><<<blocks, 32 * kWarps, smem_bytes<HD, RB>(p.a), s>>>(p);
    count_launch();
    return cudaGetLastError();
}

template <int HD, bool BF, int RB>
cudaError_t resident(int* blocks) {
    static std::atomic<int> held{0};       // by registers (shared memory holds as many)
    *blocks = held.load();
    if (*blocks > 0) return cudaSuccess;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, k_decode<HD, BF, RB>,
                                                                        32 * kWarps, kDecodeSmem<HD, RB>);
    if (e == cudaSuccess) held.store(*blocks);
    return e;
}

}  // namespace

cudaError_t launch_decode(const DecodeArgs& p, cudaStream_t s) {
    const bool one = p.row_blocks == 1;
    if (p.a.d <= 64)
        return p.a.bf16 ? (one ? launch<64, true, 1>(p, s) : launch<64, true, 2>(p, s))
                        : (one ? launch<64, false, 1>(p, s) : launch<64, false, 2>(p, s));
    return p.a.bf16 ? (one ? launch<128, true, 1>(p, s) : launch<128, true, 2>(p, s))
                    : (one ? launch<128, false, 1>(p, s) : launch<128, false, 2>(p, s));
}

cudaError_t decode_resident(const Args& a, int row_blocks, int* blocks) {
    const bool one = row_blocks == 1;
    if (a.d <= 64)
        return a.bf16 ? (one ? resident<64, true, 1>(blocks) : resident<64, true, 2>(blocks))
                      : (one ? resident<64, false, 1>(blocks) : resident<64, false, 2>(blocks));
    return a.bf16 ? (one ? resident<128, true, 1>(blocks) : resident<128, true, 2>(blocks))
                  : (one ? resident<128, false, 1>(blocks) : resident<128, false, 2>(blocks));
}

}  // namespace attn
}  // namespace fs
