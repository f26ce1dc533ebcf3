// Tree attention, many query rows per key head, on the tensor cores.
//
// A block streams the keys of its share in tiles of 64 through two streams of scores:
//   S_t = Q_t K^T (TMEM), P = 2^{x - ref} in 16 bits in TMEM, O_t += P V (TMEM),
// either two tiles of 128 query rows that share every key tile (ROWS), or, where there are
// 128 rows or fewer, one tile of rows whose key tiles go to the streams in turn (KEYS), joined at
// the end; so the softmax of one stream runs beside the products of the other.  64 rows or
// fewer (HALF) lie 16 by 16 in the four quarters of the tile: each of its four warps then has
// some, on a scheduler of its own, and half the work.
//
// Pages come by tensor copies, a page (or 64 keys of one) at a time; an entry without a
// page is copied from beyond the end of the pool, which gives zeros.  Keys and values in 16
// bits land as operand tiles.  Those in 8 bits land as they are, and four warps widen them to
// float16 (exact).  Scales stay in float32:
//   x_ij = q_i . code_j (scale2 ks_j) + log2 vs_j,   P_ij = 2^{x_ij - ref_i},
//   O_i = sum_j P_ij code_j,   sum_i = sum_j P_ij / vs_j.
// Where the scales are so far apart that P_ij could be below float32's numbers and P_ij / vs_j still
// count (rows of zeros, whose scale is 2^-89, beside others), the sum is that of the terms'
// own exponentials, 2^{x_ij - log2 vs_j - ref_i}: those tiles are weighed by a loop of their own.
// Queries in bfloat16 become float16 for that, times a power of two (query_shift) that their scores are
// divided by: one for the block where its rows are alike, else one for each.
//
// A softmax thread holds 16 keys of each of 4 rows (the 16 x 256-bit form of TMEM loads), not
// a row: the scales of its keys are then 24 loads of 8 bytes instead of 48 of 16 that
// every lane reads alike, which took most of the shared memory's time.
//
// Weights go into the products in one 16-bit part: TMEM has no columns for a second.
//
// Bound: in 16 bits by memory with 64 rows (DRAM at 81 % of its peak), with 256 by the chain of
// products and softmax (the tensor pipe is busy for 47 %).  In 8 bits a tile takes nearly as long as
// one of 16 bits, 0.7 us, with half the bytes: a tile is copied, widened, multiplied, weighed and
// multiplied again, each by other warps that wait for the last ones; with 256 rows the weighing alone
// is the longest.
// Measured, 8 key heads of 128, 32 heads: 19 x 16 tokens, 8192 keys: bfloat16 99 us, 6.5 TB/s
// (0.96 of the measured copy rate), e4m3 92 us, 3.6 TB/s; 19 x 64 tokens, 4096 keys: bfloat16 72 us,
// 1130 TFLOP/s and 4.8 TB/s, e4m3 101 us, 804 TFLOP/s.
#include "fs_tree.cuh"

#include <type_traits>

namespace fs {
namespace tree {

namespace {

using namespace fs::attn;
using kv::HELD_16;
using kv::HELD_E4M3;
using kv::HELD_I8;

constexpr int kSoftWarps = 8;              // 4 per stream
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr int kMma0 = kSoftWarps, kFit0 = kSoftWarps + 2;
enum Mode : int { ROWS = 0, KEYS = 1, HALF = 2 };
constexpr int kKeys = kTcKeys;
constexpr float kRefSlack = 8.f;
// values that may not be finite are looked through for that (whole numbers are)
template <int HELD>
constexpr bool kLooks = HELD != HELD_I8;
// tiles that the tree's keys may lie in
constexpr int kMixed = (kv::kMaxTree + kKeys - 2) / kKeys + 1;

template <int HD, int HELD, int MODE>
struct Tc {
    static constexpr bool Q8 = HELD != HELD_16;
    static constexpr bool kAlternate = MODE != ROWS;     // key tiles to the streams in turn
    // Half of the warps fit keys, half values, two warps to a tile.  HALF leaves the registers for
    // more, which take the tiles in turn: a tile takes a warp as long as its waits and latencies do,
    // whatever its share of it.
    static constexpr int kFitWarps = Q8 && MODE == HALF ? 8 : 4, kGroups = kFitWarps / 4, kFitters = 64;
    static constexpr int kCopy = kFit0 + kFitWarps;      // two warps: one copies keys, one values
    static constexpr int kThreads = 32 * (kCopy + 2);
    // HALF: products of 64 rows, whose rows 16 q .. 16 q + 15 are in lanes 32 q .. 32 q + 15
    __device__ static constexpr uint32_t tile_of(uint32_t idesc) {
        return MODE == HALF ? (idesc & ~(31u << 24)) | ((64u >> 4) << 24) : idesc;
    }
    static constexpr int kQuarter = MODE == HALF ? 16 : 32;     // rows of a softmax warp
    static constexpr int kChunks = HD / 64;
    static constexpr int kChunkBytes = kKeys * 128;               // 64 elements of each key
    static constexpr int kSlotBytes = kChunks * kChunkBytes;      // a tile of keys, or of values
    static constexpr int kQChunk = MODE == HALF ? CHUNK_BYTES / 2 : CHUNK_BYTES;     // 64 or 128 rows
    static constexpr int kQBytes = kChunks * kQChunk;
    static constexpr int kQTiles = kAlternate ? 1 : 2;
    static constexpr int kRows = 4 * kQuarter * kQTiles;
    static constexpr int kRing = Q8 ? (HD == 64 ? 4 : 3) : HD == 64 ? 8 : 4;     // tiles of each
    // Alternating streams that wait for the copies themselves (16 bits): a slot's tiles are all of
    // one stream, which waits for them in their order.  (Copies land in any: with 5 slots a
    // stream could find a slot's barrier still before the other stream's tile, take it for past
    // its own, and have the slot asked for again with a copy under way, a fault.  Widened
    // tiles are handed on in order.)
    static_assert(!kAlternate || Q8 || kRing % 2 == 0, "slots of one stream");
    static constexpr int kRaw = !Q8 ? 0 : HD == 64 ? 8 : MODE == HALF ? 6 : MODE == KEYS ? 5 : 3;    // as they land
    static_assert(kRaw % kGroups == 0, "slots of one group, which waits for them in their order");
    static constexpr int kRawBytes = kKeys * HD;
    // Descriptions of tiles are kept while the softmax may read them: it is behind the tile
    // that a slot was last used for by up to 3 (alternating streams: 5, with two groups 6), and
    // 8-bit tiles are described when they are asked for, kRaw before that.
    static constexpr int kScales = kRing + (!kAlternate ? 3 : kGroups == 1 ? 5 : 7);
    static constexpr int kBits = kScales + kRaw;
    __host__ __device__ static constexpr uint32_t S(int t) { return 256 * t; }
    __host__ __device__ static constexpr uint32_t P(int t) { return S(t) + kKeys; }    // two of 32 columns
    __host__ __device__ static constexpr uint32_t O(int t) { return P(t) + kKeys; }
    static_assert(2 * kKeys + HD <= 256, "TMEM");
};

// What the softmax needs to know of a tile.
struct TileBits {
    uint32_t counted[2];
    uint8_t poison[kKeys];       // of the tree's keys
};
struct TileScales {
    float kc[kKeys], lv[kKeys], iv[kKeys];   // of the scores; log2 and inverse of the value scale
    int odd[2], pad[2];                      // of 32 keys each: scales apart, or keys of the tree
};
struct TcBars {
    uint64_t full[2][8], free_raw[2][8];     // copies landed; 8 bits: the ring they land in
    uint64_t ready[2][8], empty[2][8];       // 8 bits: widened tiles; operand tiles done with
    // Values of the tiles with keys of the tree (the block's last), each of which has barriers of its
    // own: in 16 bits for having landed, and for having been looked through.  (The softmax does not
    // wait for values otherwise: at the barrier of a slot that the other stream's tile had before,
    // it could find that tile not there yet, take it for this one and read flags not written.)
    uint64_t last[kMixed], looked[kMixed];
    uint64_t sfull[2], sfree[2], pfull[2][2], pfree[2][2], drain[2];
    uint32_t tmem, pad;
};

template <int HD, int HELD, int MODE>
struct Smem {
    using C = Tc<HD, HELD, MODE>;
    static constexpr int q = 0;
    static constexpr int ring = q + C::kQTiles * C::kQBytes;                  // [keys, values][slot]
    static constexpr int raw = ring + 2 * C::kRing * C::kSlotBytes;           // [keys, values][slot][key][HD]
    static constexpr int raw_scale = raw + 2 * C::kRaw * C::kRawBytes;        // [slot][keys, values][key]
    static constexpr int scales = raw_scale + C::kRaw * 2 * kKeys * 4;
    static constexpr int bits = scales + (C::Q8 ? C::kScales * (int)sizeof(TileScales) : 0);
    static constexpr int words = bits + C::kBits * (int)sizeof(TileBits);     // [row's token][kTreeWords]
    static constexpr int join = words + C::kRows * 4 * kTreeWords;            // [ref, sum][stream][row]
    static constexpr int parents = join;                                      // (done with before the join)
    static constexpr int bars = join + (C::kAlternate ? 4 * 4 * 128 : 4 * kv::kMaxTree);
    static_assert(4 * 4 * 128 >= 4 * kv::kMaxTree, "parents");
    static constexpr int shift = bars + (int)sizeof(TcBars);                  // of the queries, by warps: [most, least]
    static constexpr int down = shift + 2 * 4 * kSoftWarps;                   // [row]: what scores are multiplied by
    static constexpr int bytes = down + (C::Q8 ? 4 * C::kRows : 0);
    static_assert(bits % 16 == 0 && bars % 8 == 0, "alignment");
    static_assert(1024 + bytes <= kSmemLimit, "shared memory");
};

__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 x;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at)
                 : "memory");
    return x;
}
__device__ __forceinline__ void sts16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// 16 lanes x 64 columns (16 x 256-bit form): thread t gets, for i = 0..7, columns 8 i + 2 (t % 4) +
// {0, 1} of lane t / 4 (v[4 i], v[4 i + 1]) and of lane t / 4 + 8 (v[4 i + 2], v[4 i + 3])
__device__ __forceinline__ void tmem_ld16x64(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]),
          "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]),
          "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]),
          "=f"(v[31])
        : "r"(taddr));
}
// 16 lanes x 32 columns (16 x 128-bit form): column 4 i + t % 4 of lane t / 4 (v[2 i]) and of
// lane t / 4 + 8 (v[2 i + 1])
__device__ __forceinline__ void tmem_st16x32(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15])
        : "memory");
}

// D[tmem] = A * B^T over the d elements, chunks of 64 a turn (as mma_over_d)
template <int A_CHUNK, int B_CHUNK>
__device__ __forceinline__ void mma_over_chunks(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, int chunks) {
#pragma unroll 1
    for (int x = 0; x < chunks; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y)
            mma_f16(d_tmem, a + (uint64_t)(x * (A_CHUNK >> 4) + 2 * y), b + (uint64_t)(x * (B_CHUNK >> 4) + 2 * y),
                    idesc, x != 0 || y != 0);
}

// whether 16 bytes hold an element that is not finite
template <int HELD, bool BF>
__device__ __forceinline__ bool nonfinite16(const uint4& x) {
    if (HELD == HELD_I8) return false;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (HELD == HELD_E4M3) {
            bad |= (((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
        } else {
            constexpr uint32_t kExp = BF ? 0x7f80u : 0x7c00u;
            bad |= (w[k] & kExp) == kExp || (w[k] >> 16 & kExp) == kExp;
        }
    }
    return bad;
}

// Queries in bfloat16 beside an 8-bit cache: rows whose largest elements are within 2^12 of the block's
// take its power of two, which their scores are divided by with the keys' scales; in a block with
// others each row has its own, and its scores take a factor more.
__device__ __forceinline__ bool apart_rows(int most, int least) { return most - least > 12; }
__device__ __forceinline__ void block_shift(const int* shift, int& most, int& least) {
#pragma unroll
    for (int k = 0; k < kSoftWarps; ++k) {
        most = max(most, shift[k]);
        least = min(least, shift[kSoftWarps + k]);
    }
}

// A block's share of the work.
struct Share {
    int b, kh, ctx, end, tile0, nt;
    __device__ __forceinline__ int key_of(int j) const { return (tile0 + j) * kKeys; }
    // first tile with keys of the tree, or behind the end
    __device__ __forceinline__ int mixed_from() const { return min(max(ctx / kKeys - tile0, 0), nt); }
};

// The copying warps, of keys (KV = 0, with what describes a tile) and values (1): they and the
// rings they fill are apart, as keys leave theirs two or three tiles before the values do.
template <int HD, int HELD, int MODE, int KV>
__device__ __forceinline__ void copy_tiles(const TcArgs& P, const Share& w, uint8_t* smem, TcBars& bar) {
    using C = Tc<HD, HELD, MODE>;
    using M = Smem<HD, HELD, MODE>;
    constexpr int kSlots = C::Q8 ? C::kRaw : C::kRing;
    const Args& a = P.a;
    const int lane = threadIdx.x & 31;
    // A lane to each copy: rows of a page, 64 elements wide (16 bits), or scales.  One lane for
    // all of them took 700 cycles a tile with pages of 64 and their scales, 1500 with pages of 16.
    const int rows = min(kKeys, 1 << a.c.log_page), copies = kKeys / rows;
    const int piece = lane & (copies - 1), part = lane / copies;
    const CUtensorMap* const map = KV ? &P.v : &P.k;
    const auto load_entry = [&](int j) {
        // of the tile's keys 8 (lane & 7) on
        const int i = (w.key_of(j) + 8 * (lane & 7)) >> a.c.log_page;
        int x = -1;
        if (i < a.c.table_pages)
            asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(x) : "l"(a.c.table + w.b * a.c.table_stride + i));
        return x;
    };
    const kv::Pool& scaled = part == 0 ? a.c.k : a.c.v;
    const float* scale = scaled.scale + w.kh * scaled.s_head;
    const int64_t s_page = scaled.s_page;
    const uint32_t first_of = rows == 64 ? 1u : rows == 32 ? 0x11u : rows == 16 ? 0x55u : 0xffu;
    int entry = load_entry(0), entry2 = load_entry(1), bits = 0, asked = 0;
    const int mixed_from = w.mixed_from();
    Ring r;
#pragma unroll 1
    for (; asked < w.nt; ++asked) {
        const int key0 = w.key_of(asked), key = key0 + 8 * (lane & 7);
        const bool on = (unsigned)entry < a.c.pages && key < w.end;
        const int page = on ? entry : (int)a.c.pages;          // (one behind the last: zeros)
        entry = entry2;
        entry2 = load_entry(asked + 2);
        // the other warps' barriers are not needed before the ring is full
        if (asked == min(w.nt, kSlots)) {
            __syncthreads();
        }
        if (asked >= kSlots &&
            !warp_wait((C::Q8 ? bar.free_raw[KV] : bar.empty[KV]) + r.slot, r.phase ^ 1u, a.err,
                       ERR_TIMEOUT_PRODUCER))
            break;
        const uint32_t pages = __ballot_sync(0xffffffffu, on) & 255u;
        uint64_t* const full = !C::Q8 && KV == 1 && asked >= mixed_from ? &bar.last[asked - mixed_from]
                                                                       : &bar.full[KV][r.slot];
        uint32_t bytes = C::Q8 ? C::kRawBytes : C::kSlotBytes;
        if (KV == 0) {
            // keys that count: a bit for each 8, spread; the last of them may end among their 8
            uint32_t lo = ((pages & 15u) * 0x00204081u & 0x01010101u) * 255u;
            uint32_t hi = ((pages >> 4) * 0x00204081u & 0x01010101u) * 255u;
            const int left = w.end - key0;
            if (left < 32) lo &= (1u << left) - 1u;
            if (left < 64) hi &= left <= 32 ? 0u : (1u << (left - 32)) - 1u;
            if (lane == 0)
                *reinterpret_cast<uint2*>(reinterpret_cast<TileBits*>(smem + M::bits)[bits].counted) =
                    make_uint2(lo, hi);
            // scales, only where there is a page
            if (C::Q8) bytes += 2 * 4 * rows * __popc(pages & first_of);
            if (++bits == C::kBits) bits = 0;
        }
        const int pg = __shfl_sync(0xffffffffu, page, piece * rows >> 3);
        const int slot = a.c.slot_of(key0 + piece * rows);
        if (lane == 0) mbar_arrive_expect_tx(full, bytes);
        __syncwarp();
        if (C::Q8) {
            if (part == 0)
                tma_load(smem + M::raw + (KV * C::kRaw + r.slot) * C::kRawBytes + piece * rows * HD, map, 0, slot,
                         w.kh, pg, full);
            if (KV == 0 && part < 2 && pages >> (piece * rows >> 3) & 1) {
                float* s = reinterpret_cast<float*>(smem + M::raw_scale) + r.slot * 2 * kKeys + part * kKeys +
                           piece * rows;
                bulk_g2s(s, scale + pg * s_page + slot, 4 * rows, full);
            }
        } else if (part < C::kChunks) {
            tma_load(smem + M::ring + (KV * C::kRing + r.slot) * C::kSlotBytes + part * C::kChunkBytes +
                         piece * rows * 128,
                     map, 64 * part, slot, w.kh, pg, full);
        }
        __syncwarp();
        r.step(1, kSlots);
    }
    if (w.nt <= kSlots) __syncthreads();
    // every copy lands before the block can exit, also where a wait above ran out
    const int plain = !C::Q8 && KV == 1 ? min(asked, mixed_from) : asked;
    for (int x = 0; x < min(plain, kSlots); ++x)
        warp_wait(&bar.full[KV][x], (plain - 1 - x) / kSlots & 1, a.err, ERR_TIMEOUT_PRODUCER);   // the slot's last
    for (int x = plain; x < asked; ++x) warp_wait(&bar.last[x - mixed_from], 0, a.err, ERR_TIMEOUT_PRODUCER);
}

// The fitting warps of keys (KV = 0) or values (1).  8 bits: every tile is widened into an
// operand tile.  16 bits: of the values, tiles with keys of the tree are looked through.
template <int HD, int HELD, bool BF, int MODE, int KV>
__device__ __forceinline__ void fit_tiles(const TcArgs& P, const Share& w, uint8_t* smem, TcBars& bar, int tid,
                                          int group, float mul) {
    using C = Tc<HD, HELD, MODE>;
    using M = Smem<HD, HELD, MODE>;
    constexpr bool Q8 = C::Q8;
    constexpr int kFitters = C::kFitters;
    constexpr int kPer = HD / (Q8 ? 16 : 8);            // 16-byte pieces of a row
    constexpr int kMine = kKeys * kPer / kFitters;      // of a thread: rows kStep apart
    constexpr int kStep = kFitters / kPer;
    if (!Q8 && KV == 0) return;
    const Args& a = P.a;
    const int lane = threadIdx.x & 31;
    const int u = tid % kPer, row0 = tid / kPer;
    const int mixed_from = w.mixed_from(), j0 = Q8 ? 0 : mixed_from;
    Ring from, to;
    to.slot = j0 % C::kRing;
    constexpr int kGroups = C::kGroups;
    int j_at = j0;
    if (Q8 && kGroups > 1) {
        j_at = group;
        from.step(group, Q8 ? C::kRaw : 1);
        to.step(group, C::kRing);
    }
    int scales = j_at % C::kScales, bits = j_at % C::kBits;
    Ring before;               // the tile before this one: they are handed on in their order
    if (kGroups > 1 && group == 0) before.step(1, C::kRing);
    // pieces of a row are in neighbouring lanes
    const auto look = [&](const uint4& x, int key0, int row, uint8_t* flags) {
        uint32_t bad = key0 + row >= w.ctx && nonfinite16<HELD, BF>(x);
#pragma unroll
        for (int o = kPer / 2; o; o >>= 1) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
        if (u == 0) flags[row] = (uint8_t)bad;
        return bad != 0;
    };
#pragma unroll 1
    for (int j = j_at; j < w.nt; j += kGroups) {
        const int key0 = w.key_of(j);
        TileBits& tb = reinterpret_cast<TileBits*>(smem + M::bits)[bits];
        // Of the tree's keys: a value row with an element that is not finite is zeroed, and told
        // to the softmax (0 * NaN would reach the rows that do not see it).  Rows behind the
        // end may hold anything: they are zeroed too.
        const bool mixed = j >= mixed_from;
        const uint32_t slot = smem_u32(smem) + M::ring + (KV * C::kRing + to.slot) * C::kSlotBytes;
        if (Q8) {
            if (!warp_wait(&bar.full[KV][from.slot], from.phase, a.err, ERR_TIMEOUT_PRODUCER)) return;
            const uint32_t raw = smem_u32(smem) + M::raw + (KV * C::kRaw + from.slot) * C::kRawBytes + 16 * tid;
            uint4 x[kMine];
#pragma unroll
            for (int i = 0; i < kMine; ++i) x[i] = lds16(raw + i * (16 * kFitters));
            if (mixed) {
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const int row = row0 + i * kStep;
                    const bool out = key0 + row >= w.end;
                    if (out) x[i] = make_uint4(0, 0, 0, 0);
                    if (KV == 1 && kLooks<HELD> && look(x[i], key0, row, tb.poison))
                        x[i] = make_uint4(0, 0, 0, 0);
                }
            }
            float ks = 0.f, vs = 0.f;              // (anything where there is no page)
            uint32_t counted = 0;
            const bool scaled = KV == 0 && tid < kKeys;
            if (scaled) {
                const float* s = reinterpret_cast<const float*>(smem + M::raw_scale) + from.slot * 2 * kKeys + tid;
                ks = s[0];
                vs = s[kKeys];
                counted = tb.counted[tid >> 5];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.free_raw[KV][from.slot]);
            if (j >= C::kRing && !warp_wait(&bar.empty[KV][to.slot], to.phase ^ 1u, a.err, ERR_TIMEOUT_PRODUCER))
                return;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int row = row0 + i * kStep;
                constexpr int kHeld = HELD == HELD_16 ? HELD_I8 : HELD;
                uint32_t y[8];
                kv::widen4<kHeld>(x[i].x, y[0], y[1]);
                kv::widen4<kHeld>(x[i].y, y[2], y[3]);
                kv::widen4<kHeld>(x[i].z, y[4], y[5]);
                kv::widen4<kHeld>(x[i].w, y[6], y[7]);
                const uint32_t at = slot + (u >> 2) * C::kChunkBytes;
                // the second 64 elements' lanes store their halves the other way round: the same
                // units of both chunks are in the same banks
                const bool turn = HD == 128 && u >= 4;
                const int e = (u & 3) * 16 + (turn ? 8 : 0);
                sts16(at + swz_offset(row, e), turn ? y[4] : y[0], turn ? y[5] : y[1], turn ? y[6] : y[2],
                      turn ? y[7] : y[3]);
                sts16(at + swz_offset(row, e ^ 8), turn ? y[0] : y[4], turn ? y[1] : y[5], turn ? y[2] : y[6],
                      turn ? y[3] : y[7]);
            }
            if (scaled) {
                TileScales& ts = reinterpret_cast<TileScales*>(smem + M::scales)[scales];
                float kc, lv;
                kv::weigh(ks, vs, kc, lv);
                ts.kc[tid] = kc * mul;
                ts.lv[tid] = lv;
                ts.iv[tid] = kv::weighable(vs) ? __fdividef(1.f, vs) : 0.f;
                // P / vs is lost where P < 2^-126: 2^-62 of the sum at most while all scales so far, which a
                // reference may be from, are 2^-48 to 2^16.  The tree's keys, which not every row sees, have
                // no say in how others are summed.
                const bool on = counted >> lane & 1u;
                const bool odd = mixed || __any_sync(0xffffffffu, on && !(vs >= 0x1p-48f && vs <= 0x1p16f));
                if (lane == 0) ts.odd[tid >> 5] = odd;
            }
        } else {
            if (!warp_wait(&bar.last[j - mixed_from], 0, a.err, ERR_TIMEOUT_PRODUCER)) return;
#pragma unroll 4
            for (int i = 0; i < kMine; ++i) {
                const int row = row0 + i * kStep;
                const uint32_t at = slot + (u >> 3) * C::kChunkBytes + swz_offset(row, (u & 7) * 8);
                const bool bad = look(lds16(at), key0, row, tb.poison);
                if (bad || key0 + row >= w.end) sts16(at, 0, 0, 0, 0);
            }
        }
        fence_proxy_async_smem();
        if (kGroups > 1 && j > 0) {
            if (!warp_wait(&bar.ready[KV][before.slot], before.phase, a.err, ERR_TIMEOUT_PRODUCER)) return;
            before.step(kGroups, C::kRing);
        }
        __syncwarp();
        if (lane == 0) {
            if (Q8) mbar_arrive(&bar.ready[KV][to.slot]);
            if (kLooks<HELD> && KV == 1 && mixed) mbar_arrive(&bar.looked[j - mixed_from]);
        }
        if (Q8) from.step(kGroups, Q8 ? C::kRaw : 1);
        to.step(kGroups, C::kRing);
        scales += kGroups;
        if (scales >= C::kScales) scales -= C::kScales;
        bits += kGroups;
        if (bits >= C::kBits) bits -= C::kBits;
    }
}

template <int HD, int HELD, bool BF, int MODE>
__global__ void __launch_bounds__(Tc<HD, HELD, MODE>::kThreads, 1) k_tree_tc(const __grid_constant__ TcArgs P) {
    using C = Tc<HD, HELD, MODE>;
    using M = Smem<HD, HELD, MODE>;
    using T = typename std::conditional<BF, __nv_bfloat16, __half>::type;
    constexpr bool Q8 = C::Q8;
    constexpr bool MB = BF && !Q8;             // products in bfloat16
    constexpr bool kAlternate = C::kAlternate;
    constexpr int NR = C::kRing, kCopy = C::kCopy, kFitters = C::kFitters;
    constexpr int kQuarter = C::kQuarter, kLaneRows = kQuarter / 8;     // rows of a lane: 8 apart
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    const Args& a = P.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    TcBars& bar = *reinterpret_cast<TcBars*>(smem + M::bars);
    uint32_t* sWords = reinterpret_cast<uint32_t*>(smem + M::words);
    int* sShift = reinterpret_cast<int*>(smem + M::shift);
    float* sDown = reinterpret_cast<float*>(smem + M::down);
    int* sParents = reinterpret_cast<int*>(smem + M::parents);

    int blk = blockIdx.x;
    const int split = blk % P.splits;
    blk /= P.splits;
    const int group = blk % P.groups;
    blk /= P.groups;
    Share w;
    w.kh = blk % a.c.G;
    w.b = blk / a.c.G;
    const int b = w.b, kh = w.kh;
    const int ctx = w.ctx = context(a, b);
    w.end = min(ctx + a.n, a.c.reach());
    const int nt_all = (w.end + kKeys - 1) / kKeys;
    const int per = (nt_all + P.splits - 1) / P.splits;
    const int t0 = w.tile0 = min(nt_all, split * per);
    const int nt = w.nt = min(nt_all, t0 + per) - t0;
    const int mixed_from = w.mixed_from();
    const int rows = a.R * a.n;
    const int row0 = group * C::kRows;                 // the block's first row
    const bool two = kAlternate || row0 + 128 < rows;
    const int tok0 = row0 / a.R, tok1 = min(rows - 1, row0 + C::kRows - 1) / a.R;
    const int dsteps = (a.d + 15) >> 4;
    // warps of a stream's softmax that have rows (the others leave their rows of P as they are)
    const auto warps_of = [&](int t) {
        return min(4, (rows - row0 - (kAlternate ? 0 : 128 * t) + kQuarter - 1) / kQuarter);
    };

    if (warp >= kCopy) {
        // Their barriers are their own until the block meets: they start their copies before
        // that, and meet the block once their ring is full.
        if (lane < 8) mbar_init(&bar.full[warp - kCopy][lane], 1);
        if (warp > kCopy && lane >= 8 && lane < 8 + kMixed) mbar_init(&bar.last[lane - 8], 1);
        fence_mbar_init();
        __syncwarp();
        if (warp == kCopy)
            copy_tiles<HD, HELD, MODE, 0>(P, w, smem, bar);
        else
            copy_tiles<HD, HELD, MODE, 1>(P, w, smem, bar);
        __syncthreads();
        return;
    } else if (warp < kSoftWarps) {
        // what the block's tokens see of the tree, then their queries as operand tiles
        if (a.parents) {
            const int32_t* p = a.parents + b * a.parents_stride;
            for (int e = threadIdx.x; e < a.n; e += kSoftThreads) sParents[e] = __ldg(p + e);
            named_sync(1, kSoftThreads);
        }
        if ((int)threadIdx.x <= tok1 - tok0) {
            uint32_t x[kTreeWords];
            tree_row(a.parents ? sParents : nullptr, tok0 + threadIdx.x, x);
#pragma unroll
            for (int k = 0; k < kTreeWords; ++k) sWords[threadIdx.x * kTreeWords + k] = x[k];
        }
        named_sync(1, kSoftThreads);
        constexpr int kPieces = HD / 8;        // of a row, in neighbouring lanes
        constexpr int kMine = C::kRows * kPieces / kSoftThreads, kStep = kSoftThreads / kPieces;
        const int u = threadIdx.x % kPieces;
        uint32_t x[kMine][4];
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int all = row0 + threadIdx.x / kPieces + i * kStep;
            x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0;
            if (all < rows && 8 * u < a.d) {
                const int tok = all / a.R;
                const uint32_t* s = sWords + (tok - tok0) * kTreeWords;
                if (s[tok >> 5] >> (tok & 31) & 1u) {
                    const uint16_t* p = static_cast<const uint16_t*>(a.q.p) + b * a.q.sb + tok * a.q.st +
                                        (int64_t)(kh * a.R + all - tok * a.R) * a.q.sh + 8 * u;
                    if (a.q_vec) {
                        const uint4 y = __ldg(reinterpret_cast<const uint4*>(p));
                        x[i][0] = y.x, x[i][1] = y.y, x[i][2] = y.z, x[i][3] = y.w;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[i][k] = (uint32_t)p[2 * k] | (uint32_t)p[2 * k + 1] << 16;
                    }
                }
            }
        }
        if (Q8 && BF) {
            int up[kMine], most = -126, least = 126;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) top = finite_top(top, x[i][k]);
#pragma unroll
                for (int o = kPieces / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                up[i] = query_shift(top);
                least = min(least, up[i]);
                if (top != 0) most = max(most, up[i]);         // (rows of zeros take any)
            }
            least = __reduce_min_sync(0xffffffffu, least);
            most = __reduce_max_sync(0xffffffffu, most);
            if (lane == 0) {
                sShift[warp] = most;
                sShift[kSoftWarps + warp] = least;
            }
            named_sync(1, kSoftThreads);
            block_shift(sShift, most, least);
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int more = apart_rows(most, least) ? min(up[i] - least, 126) : 0;
                if (u == 0) sDown[threadIdx.x / kPieces + i * kStep] = two_to(-more);
#pragma unroll
                for (int k = 0; k < 4; ++k) x[i][k] = shifted_pair(x[i][k], two_to(least + more));
            }
        }
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int r = threadIdx.x / kPieces + i * kStep;
            sts16(smem_u32(smem) + M::q + (r >> 7) * C::kQBytes + (u >> 3) * C::kQChunk +
                      swz_offset(r & 127, (u & 7) * 8),
                  x[i][0], x[i][1], x[i][2], x[i][3]);
        }
        fence_proxy_async_smem();
    } else if (warp == kMma0) {
        if (lane < 16) {
            mbar_init(&bar.ready[lane >> 3][lane & 7], 2);
            mbar_init(&bar.empty[lane >> 3][lane & 7], !kAlternate && two ? 2 : 1);
            mbar_init(&bar.free_raw[lane >> 3][lane & 7], 2);
        } else if (lane < 16 + kMixed) {
            mbar_init(&bar.looked[lane - 16], 2);
        } else if (lane >= 30) {
            const int t = lane - 30;
            mbar_init(&bar.sfull[t], 1);
            const int warps = max(1, warps_of(t));
            mbar_init(&bar.sfree[t], warps);
            mbar_init(&bar.pfull[t][0], warps);
            mbar_init(&bar.pfull[t][1], warps);
            mbar_init(&bar.pfree[t][0], 1);
            mbar_init(&bar.pfree[t][1], 1);
            mbar_init(&bar.drain[t], 1);
        }
        fence_mbar_init();
    } else if (warp == kMma0 + 1) {
        tmem_alloc(&bar.tmem, 512);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;

    if (warp >= kFit0) {
        float mul = a.scale2;
        if (Q8 && BF) {
            int most = -126, least = 126;
            block_shift(sShift, most, least);
            mul *= two_to(-least);
        }
        const int tid = (threadIdx.x - 32 * kFit0) & (kFitters - 1), fit = (warp - kFit0) >> 1;
        if (fit < C::kGroups)
            fit_tiles<HD, HELD, BF, MODE, 0>(P, w, smem, bar, tid, fit, mul);
        else
            fit_tiles<HD, HELD, BF, MODE, 1>(P, w, smem, bar, tid, fit - C::kGroups, mul);
    } else if (warp >= kMma0) {
        const int t = warp - kMma0;
        const int n_mine = kAlternate ? (nt + 1 - t) / 2 : nt;
        if (n_mine > 0 && (t == 0 || two) && elect_one()) {
            constexpr int kBy = kAlternate ? 2 : 1;
            const uint32_t idS = C::tile_of(idesc_16(MB, kKeys, false)), idO = C::tile_of(idesc_16(MB, dsteps * 16, true));
            constexpr uint64_t kSlotU = C::kSlotBytes >> 4;    // descriptors count 16 bytes
            const uint64_t dQ = sdesc_sw128(smem_u32(smem + M::q)) + (kAlternate ? 0 : t) * (C::kQBytes >> 4);
            const uint64_t dK = sdesc_sw128(smem_u32(smem + M::ring));
            const uint64_t dV = sdesc_tokens(smem_u32(smem + M::ring) + NR * C::kSlotBytes, C::kChunkBytes);
            const uint32_t cS = tmem + C::S(t), cP = tmem + C::P(t), cO = tmem + C::O(t);
            uint64_t* const k_in = Q8 ? bar.ready[0] : bar.full[0];
            Ring rk, rv;
            if (kAlternate) rk.step(t, NR), rv.step(t, NR);
            bool ok = true;
            for (int j = -1; j < n_mine && ok; ++j) {
                if (j + 1 < n_mine) {
                    if (!(ok = mma_wait(a.err, k_in + rk.slot, rk.phase) &&
                               (j < 0 || mma_wait(a.err, &bar.sfree[t], j & 1))))
                        break;
                    mma_over_chunks<C::kQChunk, C::kChunkBytes>(cS, dQ, dK + rk.slot * kSlotU, idS, (dsteps + 3) / 4);
                    mma_commit(&bar.sfull[t]);
                    mma_commit(&bar.empty[0][rk.slot]);
                    rk.step(kBy, NR);
                }
                if (j < 0) continue;
                const int buf = j & 1, tile = kAlternate ? 2 * j + t : j;
                const bool own = !Q8 && tile >= mixed_from;
                uint64_t* const v_in = Q8 ? &bar.ready[1][rv.slot]
                                          : own ? &bar.looked[tile - mixed_from] : &bar.full[1][rv.slot];
                if (!(ok = mma_wait(a.err, v_in, own ? 0 : rv.phase) &&
                           mma_wait(a.err, &bar.pfull[t][buf], (j >> 1) & 1)))
                    break;
                mma_over_tokens<kKeys>(cO, cP + buf * (kKeys / 2), dV + rv.slot * kSlotU, idO, j > 0, 32);
                mma_commit(&bar.pfree[t][buf]);
                mma_commit(&bar.empty[1][rv.slot]);
                rv.step(kBy, NR);
            }
            mma_commit(&bar.drain[t]);
            mbar_wait(&bar.drain[t], 0, a.err, ERR_TIMEOUT_MMA);
        }
    } else {
        const int t = warp >> 2, quarter = warp & 3;
        const uint32_t lofs = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + C::S(t) + lofs, tP = tmem + C::P(t) + lofs, tO = tmem + C::O(t) + lofs;
        const int n_mine = quarter >= warps_of(t) ? 0 : kAlternate ? (nt + 1 - t) / 2 : nt;
        const int g = lane >> 2, t4 = lane & 3;
        const int row_t = row0 + (kAlternate ? 0 : 128 * t) + quarter * kQuarter;    // the warp's first row
        const float mul = a.scale2;                  // (8 bits: with the keys' scales)
        const uint64_t mul2 = pk(mul, mul);
        bool factors = false;                        // of the rows' scores
        if (Q8 && BF) {
            int most = -126, least = 126;
            block_shift(sShift, most, least);
            factors = apart_rows(most, least);
        }
        const float* down = sDown + (kAlternate ? 0 : 128 * t) + quarter * kQuarter + g;
        // of rows g + 8 k of the warp; a lane's part of the sum
        float ref[kLaneRows], sum[kLaneRows];
#pragma unroll
        for (int k = 0; k < kLaneRows; ++k) {
            ref[k] = -INFINITY;
            sum[k] = 0.f;
        }
        // A tile of the stream, scored: P and the sums; false if a wait ran out.  Beside an 8-bit cache `plain`
        // takes tiles whose keys all rows see, in blocks without factors and with scales near one another.
        bool apart = false;                          // scales that were not, so far
        const auto weigh_tile = [&](auto plain, int j, int tile) -> bool {
            constexpr bool kPlain = decltype(plain)::value;
            const int key0 = (t0 + tile) * kKeys;
            // v[32 h + 4 i + e]: column 8 i + 2 t4 + (e & 1) of row g + 8 (2 h + (e >> 1))
            float v[16 * kLaneRows];
            tmem_ld16x64(tS, v);
            if (kLaneRows > 2) tmem_ld16x64(tS + (16u << 16), v + (kLaneRows > 2 ? 32 : 0));
            const TileBits& tb = reinterpret_cast<const TileBits*>(smem + M::bits)[tile % C::kBits];
            const TileScales& ts = reinterpret_cast<const TileScales*>(smem + M::scales)[tile % C::kScales];
            uint64_t kc[Q8 ? 8 : 1], lv[Q8 ? 8 : 1];
            if (Q8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    kc[Q8 ? i : 0] = *reinterpret_cast<const uint64_t*>(ts.kc + 8 * i + 2 * t4);
                    lv[Q8 ? i : 0] = *reinterpret_cast<const uint64_t*>(ts.lv + 8 * i + 2 * t4);
                }
            }
            const uint2 counted = *reinterpret_cast<const uint2*>(tb.counted);
            tmem_wait_ld();
            tmem_reg_fence(v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.sfree[t]);
            if (Q8 && BF && !kPlain && factors) {
#pragma unroll
                for (int k = 0; k < kLaneRows; ++k) {
                    const float f = down[8 * k];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float* x = v + 32 * (k >> 1) + 4 * i + 2 * (k & 1);
                        upk(mul2f(pk(x[0], x[1]), pk(f, f)), x[0], x[1]);
                    }
                }
            }
            if (Q8) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int k = 0; k < kLaneRows; ++k) {
                        float* x = v + 32 * (k >> 1) + 4 * i + 2 * (k & 1);
                        upk(fma2(pk(x[0], x[1]), kc[Q8 ? i : 0], lv[Q8 ? i : 0]), x[0], x[1]);
                    }
            }
            const bool mixed = !kPlain && tile >= mixed_from;
            if (mixed || (counted.x & counted.y) != 0xffffffffu) {
                uint32_t bad[2] = {0, 0};
                if (kLooks<HELD> && mixed) {
                    // the values' check may come behind the scores
                    if (!warp_wait(&bar.looked[tile - mixed_from], 0, a.err, ERR_TIMEOUT_EPILOGUE)) return false;
#pragma unroll
                    for (int x = 0; x < 2; ++x) bad[x] = __ballot_sync(0xffffffffu, tb.poison[32 * x + lane] != 0);
                }
#pragma unroll
                for (int k = 0; k < kLaneRows; ++k) {
                    uint32_t sees[2] = {counted.x, counted.y};
                    if (mixed) {
                        const int tok = min(row_t + g + 8 * k, rows - 1) / a.R;
                        const uint32_t* words = sWords + (tok - tok0) * kTreeWords;
                        const bool there = words[tok >> 5] >> (tok & 31) & 1u;
                        sees[0] &= tree_window(words, there, key0 - ctx);
                        sees[1] &= tree_window(words, there, key0 + 32 - ctx);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int at = (8 * i & 31) + 2 * t4 + e;
                            float& x = v[32 * (k >> 1) + 4 * i + 2 * (k & 1) + e];
                            if (bad[i >> 2] >> at & 1u) x = __uint_as_float(0x7fc00000u);
                            if (!(sees[i >> 2] >> at & 1u)) x = -INFINITY;
                        }
                }
            }
            float m[kLaneRows];                // over this lane's keys
            bool moves = false;
#pragma unroll
            for (int k = 0; k < kLaneRows; ++k) {
                const float* x = v + 32 * (k >> 1) + 2 * (k & 1);
                float m0 = fmaxf(x[0], x[1]), m1 = fmaxf(x[4], x[5]);
#pragma unroll
                for (int i = 2; i < 8; i += 2) {
                    m0 = max3(m0, x[4 * i], x[4 * i + 1]);
                    m1 = max3(m1, x[4 * i + 4], x[4 * i + 5]);
                }
                m[k] = fmaxf(m0, m1);
                if (!Q8) m[k] *= mul;
                moves |= m[k] > ref[k] + kRefSlack;
            }
            const int buf = j & 1;
            // Rarely: references move, and O and the sums with them.
            if (__any_sync(0xffffffffu, moves)) {
                float f = 1.f;                 // of row `lane`
#pragma unroll
                for (int k = 0; k < kLaneRows; ++k) {
                    float top = fmaxf(m[k], __shfl_xor_sync(0xffffffffu, m[k], 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    float alpha = 1.f;
                    if (top > ref[k] + kRefSlack) {
                        if (Q8) top = ceilf(top);
                        // (up to its first counted key a row's sum and O are zero)
                        if (ref[k] != -INFINITY) {
                            alpha = ex2(ref[k] - top);
                            sum[k] = Q8 ? kv::moved_sum(sum[k], ref[k] - top) : sum[k] * alpha;
                        }
                        ref[k] = top;
                    }
                    const float x = __shfl_sync(0xffffffffu, alpha, 4 * (lane & 7));
                    f = lane >> 3 == k ? x : f;
                }
                if (__any_sync(0xffffffffu, f != 1.f)) {
                    // O is still once the products of tile j - 1 are done (j > 0 here)
                    if (!warp_wait(&bar.pfree[t][buf ^ 1], ((j - 1) >> 1) & 1, a.err, ERR_TIMEOUT_EPILOGUE))
                        return false;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < dsteps * 16; c += 16) {
                        float o[16];
                        tmem_ld16(tO + c, o);
                        tmem_wait_ld();
                        tmem_reg_fence(o);
                        uint32_t y[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(o[e] * f);
                        tmem_st16(tO + c, y);
                    }
                }
            }
            uint64_t base2[kLaneRows];
#pragma unroll
            for (int k = 0; k < kLaneRows; ++k) {
                const float base = kProbShift<MB> - (ref[k] == -INFINITY ? 0.f : ref[k]);
                base2[k] = pk(base, base);
            }
            uint64_t s[kLaneRows];
#pragma unroll
            for (int k = 0; k < kLaneRows; ++k) s[k] = 0;
            if (Q8 && !kPlain && apart) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 l = *reinterpret_cast<const float2*>(ts.lv + 8 * i + 2 * t4);
#pragma unroll
                    for (int k = 0; k < kLaneRows; ++k) {
                        const float* x = v + 32 * (k >> 1) + 4 * i + 2 * (k & 1);
                        float e0, e1;
                        upk(add2(pk(x[0] - l.x, x[1] - l.y), base2[k]), e0, e1);
                        s[k] = add2(s[k], pk(ex2(e0), ex2(e1)));
                    }
                }
            }
            uint32_t p[8 * kLaneRows];         // p[16 h + 2 i + (k & 1)]
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint64_t iv =
                    Q8 && (kPlain || !apart) ? *reinterpret_cast<const uint64_t*>(ts.iv + 8 * i + 2 * t4) : 0;
#pragma unroll
                for (int k = 0; k < kLaneRows; ++k) {
                    const float* x = v + 32 * (k >> 1) + 4 * i + 2 * (k & 1);
                    float e0, e1;
                    upk(Q8 ? add2(pk(x[0], x[1]), base2[k]) : fma2(pk(x[0], x[1]), mul2, base2[k]), e0, e1);
                    e0 = ex2(e0);
                    e1 = ex2(e1);
                    s[k] = Q8 ? fma2(pk(e0, e1), iv, s[k]) : add2(s[k], pk(e0, e1));
                    p[16 * (k >> 1) + 2 * i + (k & 1)] = pack16<MB>(e0, e1);
                }
            }
            // this buffer's last P, of tile j - 2, was read when S of this tile was done
            tmem_st16x32(tP + buf * (kKeys / 2), p);
            if (kLaneRows > 2) tmem_st16x32(tP + buf * (kKeys / 2) + (16u << 16), p + (kLaneRows > 2 ? 16 : 0));
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.pfull[t][buf]);
#pragma unroll
            for (int k = 0; k < kLaneRows; ++k) {
                float f0, f1;
                upk(s[k], f0, f1);
                sum[k] += f0 + f1;
            }
            return true;
        };
        // Beside an 8-bit cache the plain tiles, as long as they come, then the others, in two loops.  (All
        // in one, or each of two bodies by a test in one loop, took the registers that keep a tile's stages
        // side by side: 19 x 64 tokens, 4096 e4m3 keys 125 and 105 us for 101, 32 x 16 tokens 167 for
        // 159.)
        bool ok = true;
        int j = 0;
        const auto odd = [&](int tile) {
            const int2 x = *reinterpret_cast<const int2*>(
                reinterpret_cast<const TileScales*>(smem + M::scales)[tile % C::kScales].odd);
            return __any_sync(0xffffffffu, (x.x | x.y) != 0) != 0;
        };
        for (; Q8 && !factors && j < n_mine; ++j) {
            const int tile = kAlternate ? 2 * j + t : j;
            if (!(ok = warp_wait(&bar.sfull[t], j & 1, a.err, ERR_TIMEOUT_EPILOGUE))) break;
            if (odd(tile)) break;
            tc_fence_after();
            if (!(ok = weigh_tile(std::integral_constant<bool, Q8>(), j, tile))) break;
        }
        for (; j < n_mine && ok; ++j) {
            const int tile = kAlternate ? 2 * j + t : j;
            if (!(ok = warp_wait(&bar.sfull[t], j & 1, a.err, ERR_TIMEOUT_EPILOGUE))) break;
            tc_fence_after();
            if (Q8) apart = apart || odd(tile);
            ok = weigh_tile(std::false_type(), j, tile);
        }
        if (n_mine > 0 && ok) {
            const int j = n_mine - 1;
            ok = warp_wait(&bar.pfree[t][j & 1], (j >> 1) & 1, a.err, ERR_TIMEOUT_EPILOGUE);
        }
        tc_fence_after();
        // from here on a row to a thread
        float total = 0.f, top = -INFINITY;
#pragma unroll
        for (int k = 0; k < kLaneRows; ++k) {
            sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
            sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
            const float x = __shfl_sync(0xffffffffu, sum[k], 4 * (lane & 7));
            const float y = __shfl_sync(0xffffffffu, ref[k], 4 * (lane & 7));
            if (lane >> 3 == k) {
                total = x;
                top = y;
            }
        }
        const int r = quarter * 32 + lane;                 // of the stream's tile
        const int all = min(row_t + lane, rows - 1);
        const bool live = lane < kQuarter && row_t + lane < rows;
        const int tok = all / a.R, head = kh * a.R + all - tok * a.R;
        const bool there = sWords[(tok - tok0) * kTreeWords + (tok >> 5)] >> (tok & 31) & 1u;
        // Alternating streams: both sums of the row, each stream then half of its columns
        float f[2] = {1.f, 0.f};
        int c0 = 0, c1 = dsteps * 16;
        if (kAlternate) {
            float* join = reinterpret_cast<float*>(smem + M::join);
            join[t * 128 + r] = top;
            join[256 + t * 128 + r] = total;
            tc_fence_before();
            named_sync(1, kSoftThreads);
            tc_fence_after();
            top = fmaxf(join[r], join[128 + r]);
            const float base = top == -INFINITY ? 0.f : top;
            total = 0.f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float by = join[128 * x + r] - base, part = join[256 + 128 * x + r];
                f[x] = ex2(by);
                total = Q8 ? total + kv::moved_sum(part, by) : fmaf(f[x], part, total);
            }
            c0 = t ? (dsteps + 1) / 2 * 16 : 0;
            c1 = t ? dsteps * 16 : (dsteps + 1) / 2 * 16;
        }
        const bool none = total == 0.f || !there;
        const float inv = none ? 0.f : 1.f / total;
        const int64_t row = ((int64_t)b * a.H + head) * a.n + tok;
        if (live && (!kAlternate || t == 0)) {
            const float lse2 = none ? -INFINITY
                               : Q8 ? kv::log_sum(top - kProbShift<MB>, total)
                                    : top - kProbShift<MB> + lg2(total);
            if (P.splits > 1)
                P.part.lse2[split * P.part.rows + row] = lse2;
            else
                a.lse[row] = lse2 * (float)kLn2;
        }
        // Each thread writes 16 elements of its row at a time.
        T* out = static_cast<T*>(a.o.p) + b * a.o.sb + tok * a.o.st + (int64_t)head * a.o.sh;
        float* part = P.splits > 1 ? P.part.out + (split * P.part.rows + row) * a.d : nullptr;
        const uint32_t o_at[2] = {tmem + C::O(kAlternate ? 0 : t) + lofs, tmem + C::O(1) + lofs};
        const int streams = kAlternate ? (nt > 1 ? 2 : nt) : nt > 0;
        const bool any = quarter < warps_of(t);
#pragma unroll 1
        for (int c = c0; c < c1 && any; c += 16) {
            __syncwarp();
            float o[16], y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = y[e] = 0.f;
            if (streams > 0) tmem_ld16(o_at[0] + c, o);
            if (kAlternate && streams > 1) tmem_ld16(o_at[1] + c, y);
            tmem_wait_ld();
            tmem_reg_fence(o);
            tmem_reg_fence(y);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                o[e] = kAlternate ? (f[0] == 0.f ? 0.f : f[0] * o[e]) + (f[1] == 0.f ? 0.f : f[1] * y[e]) : o[e];
                o[e] = none ? 0.f : o[e] * inv;
            }
            if (!live || !ok) {
                // nothing to write
            } else if (part) {
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    if (c + e < a.d)
                        *reinterpret_cast<float4*>(part + c + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            } else if (P.o_vec) {
#pragma unroll
                for (int e = 0; e < 16; e += 8)
                    if (c + e < a.d)
                        *reinterpret_cast<uint4*>(out + c + e) =
                            make_uint4(pack16<BF>(o[e], o[e + 1]), pack16<BF>(o[e + 2], o[e + 3]),
                                       pack16<BF>(o[e + 4], o[e + 5]), pack16<BF>(o[e + 6], o[e + 7]));
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (c + e < a.d) out[c + e] = from_f<T>(o[e]);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMma0 + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int HD, int HELD, bool BF, int MODE>
cudaError_t launch(const TcArgs& p, cudaStream_t s) {
    constexpr size_t bytes = 1024 + Smem<HD, HELD, MODE>::bytes;
    static std::atomic<uint64_t> ready{0};    // devices whose shared-memory limit is raised
    if (cudaError_t e = raise_smem(k_tree_tc<HD, HELD, BF, MODE>, bytes, ready); e != cudaSuccess) return e;
    const unsigned blocks = (unsigned)((int64_t)p.a.c.B * p.a.c.G * p.groups * p.splits);
    k_tree_tc<HD, HELD, BF, MODE><<<blocks, Tc<HD, HELD, MODE>::kThreads, bytes, s>>>(p);
    count_launch();
    return cudaGetLastError();
}
template <int HD, int HELD, bool BF>
cudaError_t launch_mode(const TcArgs& p, cudaStream_t s) {
    const int rows = p.a.R * p.a.n;
    if (rows > 128) return launch<HD, HELD, BF, ROWS>(p, s);
    return rows > 64 ? launch<HD, HELD, BF, KEYS>(p, s) : launch<HD, HELD, BF, HALF>(p, s);
}
template <int HD, int HELD>
cudaError_t launch_held(const TcArgs& p, cudaStream_t s) {
    return p.a.bf16 ? launch_mode<HD, HELD, true>(p, s) : launch_mode<HD, HELD, false>(p, s);
}
template <int HD>
cudaError_t launch_width(const TcArgs& p, cudaStream_t s) {
    if (p.a.c.held == HELD_16) return launch_held<HD, HELD_16>(p, s);
    return p.a.c.held == HELD_E4M3 ? launch_held<HD, HELD_E4M3>(p, s) : launch_held<HD, HELD_I8>(p, s);
}

}  // namespace

bool tc_copies(const Cache& c) {
    constexpr int64_t kFar = int64_t(1) << 39;
    if (c.pages == 0) return false;
    for (const kv::Pool* w : {&c.k, &c.v}) {
        const auto step = [&](int64_t size, int64_t s) { return size <= 1 || (s > 0 && s % 16 == 0 && s < kFar); };
        if (reinterpret_cast<uintptr_t>(w->p) % 16 || !step(2, w->token) || !step(c.G, w->head) ||
            !step(c.pages, w->page))
            return false;
        if (c.held != HELD_16 && (reinterpret_cast<uintptr_t>(w->scale) % 16 || (c.G > 1 && w->s_head % 4) ||
                                  (c.pages > 1 && w->s_page % 4)))
            return false;
    }
    return true;
}

fs_status tc_maps(TcArgs& p, bool bf16) {
    const Cache& c = p.a.c;
    const bool bytes = c.held != HELD_16;
    const uint64_t row = (uint64_t)(c.d * (bytes ? 1 : 2) + 15) / 16 * 16;
    const uint64_t dims[4] = {(uint64_t)c.d, uint64_t(1) << c.log_page, (uint64_t)c.G, c.pages};
    const uint32_t box[4] = {bytes ? (c.d <= 64 ? 64u : 128u) : 64u, (uint32_t)std::min(kKeys, 1 << c.log_page),
                             1, 1};
    for (int x = 0; x < 2; ++x) {
        const kv::Pool& w = x ? c.v : c.k;
        const uint64_t strides[3] = {(uint64_t)w.token, c.G > 1 ? (uint64_t)w.head : row,
                                     c.pages > 1 ? (uint64_t)w.page : row};
        FS_TRY(bytes ? make_tmap_4d_bytes(x ? &p.v : &p.k, w.p, dims, strides, box)
                     : make_tmap_4d(x ? &p.v : &p.k, w.p, dims, strides, box, bf16));
    }
    return FS_OK;
}

cudaError_t launch_tc(const TcArgs& p, cudaStream_t s) {
    return p.a.d <= 64 ? launch_width<64>(p, s) : launch_width<128>(p, s);
}

}  // namespace tree
}  // namespace fs
