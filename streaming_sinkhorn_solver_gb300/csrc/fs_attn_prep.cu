// Small kernels around the cross-attention kernels: the key tiles of a mask,
// the join of partial results, copies of tensors that the tensor maps cannot
// read in place, results of empty calls; and the tensor maps themselves.
#include "fs_attn_host.cuh"

namespace fs {
namespace attn {

namespace {

// One block per sequence: the bits of the counted keys of each tile, and the
// tiles that have any, in order.  A warp takes a tile per round; the rounds'
// places come from a ballot over the warps.
constexpr int kListThreads = 1024;
__global__ void __launch_bounds__(kListThreads) k_key_tiles(Args a, uint4* __restrict__ words,
                                                            int* __restrict__ list,
                                                            int* __restrict__ count, int tiles) {
    __shared__ int found[32];
    const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int end = key_end(a, b);
    const uint8_t* mask = a.mask + (int64_t)b * a.mask_stride;
    int base = 0;
    for (int t0 = 0; t0 < tiles; t0 += 32) {
        const int t = t0 + warp;
        bool any = false;
        if (t < tiles) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = t * kTile + 32 * k + lane;
                w[k] = __ballot_sync(0xffffffffu, j < end && __ldg(mask + j) != 0);
            }
            any = (w[0] | w[1] | w[2] | w[3]) != 0;
            if (lane == 0) words[(int64_t)b * tiles + t] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (lane == 0) found[warp] = any;
        __syncthreads();
        const uint32_t hit = __ballot_sync(0xffffffffu, found[lane] != 0);
        if (any && lane == 0)
            list[(int64_t)b * tiles + base + __popc(hit & ((1u << warp) - 1u))] = t;
        base += __popc(hit);
        __syncthreads();
    }
    if (threadIdx.x == 0) count[b] = base;
}

// Joins the partial rows of all splits in their order: a warp per row.
template <typename T>
__global__ void __launch_bounds__(128) k_combine(Args a, Partials part, int splits) {
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= part.rows) return;
    const int i = (int)(row % a.n);
    const int64_t bh = row / a.n;
    const int h = (int)(bh % a.H), b = (int)(bh / a.H);
    T* out = static_cast<T*>(a.o.p) + b * a.o.sb + (int64_t)i * a.o.st + h * a.o.sh;
    float top = -INFINITY;
    for (int s = lane; s < splits; s += 32) top = fmaxf(top, part.lse2[s * part.rows + row]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = top == -INFINITY ? 0.f : top;
    float total = 0.f, acc[kMaxHeadDim / 32];
#pragma unroll
    for (int e = 0; e < kMaxHeadDim / 32; ++e) acc[e] = 0.f;
    for (int s0 = 0; s0 < splits; s0 += 32) {
        const float mine = s0 + lane < splits ? ex2(part.lse2[(s0 + lane) * part.rows + row] - base) : 0.f;
        const int some = min(32, splits - s0);
#pragma unroll 4
        for (int s = 0; s < some; ++s) {
            const float w = __shfl_sync(0xffffffffu, mine, s);
            total += w;
            const float* src = part.out + ((s0 + s) * part.rows + row) * a.d;
#pragma unroll
            for (int e = 0; e < kMaxHeadDim / 32; ++e)
                if (lane + 32 * e < a.d) acc[e] = fmaf(w, src[lane + 32 * e], acc[e]);
        }
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
    for (int e = 0; e < kMaxHeadDim / 32; ++e)
        if (lane + 32 * e < a.d) out[lane + 32 * e] = from_f<T>(total == 0.f ? 0.f : acc[e] * inv);
    if (lane == 0) a.lse[row] = total == 0.f ? -INFINITY : (top + lg2(total)) * (float)kLn2;
}

// rows (b, h, token): out 0, and lse -inf where there is one
__global__ void __launch_bounds__(128) k_zero(View w, int64_t rows, int tokens, int heads, int d,
                                              float* __restrict__ lse) {
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const int t = (int)(row % tokens);
    const int h = (int)(row / tokens % heads);
    const int b = (int)(row / tokens / heads);
    uint16_t* p = static_cast<uint16_t*>(w.p) + b * w.sb + (int64_t)t * w.st + h * w.sh;
    for (int c = lane; c < d; c += 32) p[c] = 0;
    if (lse && lane == 0) lse[row] = -INFINITY;
}

__global__ void __launch_bounds__(128) k_pack(View w, uint16_t* __restrict__ to, int64_t rows, int tokens,
                                              int heads, int d, int dp) {
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);   // (b, t, h)
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const int h = (int)(row % heads);
    const int t = (int)(row / heads % tokens);
    const int b = (int)(row / heads / tokens);
    const uint16_t* p = static_cast<const uint16_t*>(w.p) + b * w.sb + (int64_t)t * w.st + h * w.sh;
    for (int c = lane; c < dp; c += 32) to[row * dp + c] = c < d ? p[c] : (uint16_t)0;
}

}  // namespace

cudaError_t launch_key_tiles(const Args& a, uint4* words, int* list, int* count, int tiles,
                             cudaStream_t s) {
    k_key_tiles<<<a.B, kListThreads, 0, s>>>(a, words, list, count, tiles);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_combine(const Args& a, const Partials& part, int splits, cudaStream_t s) {
    const unsigned blocks = (unsigned)((part.rows + 3) / 4);
    if (a.bf16)
        k_combine<__nv_bfloat16><<<blocks, 128, 0, s>>>(a, part, splits);
    else
        k_combine<__half><<<blocks, 128, 0, s>>>(a, part, splits);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_zero(const Args& a, const View& w, int tokens, int heads, float* lse, cudaStream_t s) {
    const int64_t rows = (int64_t)a.B * tokens * heads;
    if (rows == 0) return cudaSuccess;
    k_zero<<<(unsigned)((rows + 3) / 4), 128, 0, s>>>(w, rows, tokens, heads, a.d, lse);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_pack(const View& from, void* to, int B, int tokens, int heads, int d, int dp,
                        cudaStream_t s) {
    const int64_t rows = (int64_t)B * tokens * heads;
    if (rows == 0) return cudaSuccess;
    k_pack<<<(unsigned)((rows + 3) / 4), 128, 0, s>>>(from, static_cast<uint16_t*>(to), rows, tokens,
                                                      heads, d, dp);
    count_launch();
    return cudaGetLastError();
}

fs_status make_tensor_map(TensorMap& t, const View& w, int B, int tokens, int heads, int d, bool bf16,
                          int rows) {
    // (d, token, head, batch); an axis of one entry or of stride 0 has one entry
    const uint64_t row = 2 * (uint64_t)((d + 7) / 8 * 8);
    t.head = heads > 1 && w.sh != 0;
    t.batch = B > 1 && w.sb != 0;
    const uint64_t dims[4] = {(uint64_t)d, (uint64_t)tokens, t.head ? (uint64_t)heads : 1,
                              t.batch ? (uint64_t)B : 1};
    const uint64_t strides[3] = {tokens > 1 ? 2 * (uint64_t)w.st : row, t.head ? 2 * (uint64_t)w.sh : row,
                                 t.batch ? 2 * (uint64_t)w.sb : row};
    const uint32_t box[4] = {64, (uint32_t)rows, 1, 1};
    return make_tmap_4d(&t.map, w.p, dims, strides, box, bf16);
}

}  // namespace attn
}  // namespace fs
