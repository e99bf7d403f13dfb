// Attention of many query rows over the 4-bit cache on the fifth-generation
// tensor cores (tcgen05 MMAs, accumulators in tensor memory).
//
// The rows of a KV head are packed, row r = token r / group, query head
// r mod group, so that every query head shares each decoded tile.  One CTA
// takes two blocks of 128 rows and a range of key tiles of 128 positions:
//   warps 0-3, 4-7  softmax warpgroups: thread i of warpgroup g owns row i of
//                   block g, which is lane i of tensor memory; each brings in
//                   its own query row first (rotated, to fp16)
//   warp 8          issues the MMAs (one elected lane)
//   warps 9-15      decode the tiles (a value is exact in fp16).  A tile is 16
//                   pieces of work, the keys of its eight groups of 16
//                   positions, then their values, 1152 bytes each (kPer = 2:
//                   eight of twice the size), that the warps take in turn;
//                   each brings its own pieces (cp.async, four halves of a
//                   group ahead)
// Decoded tiles are K-major operands with the 128-byte swizzle.  Values are
// stored transposed, [dim][position]: two neighbouring positions share a byte,
// so the conversion of a byte gives a pair that lies side by side there, and
// the stores of a warp fall on 32 distinct banks.  A tile is decoded once for
// 256 rows.
// What bounds it: 2048 rows of 8 query heads onto 34815 positions of two KV heads
// take 428 us, 3300 clocks a tile of 256 rows, 2100 of them products (tensor pipe
// 56 %; the rest of the time the products wait for decoded tiles and for P).  Their
// operands (192 KB a tile) and the decoded stores (64 KB) share shared memory's 128
// bytes a clock, and a piece takes its warp about 1080 clocks, with or without its
// conversions, its loads or the softmax's exponentials.  Copies started by one
// lane, a barrier each, took 400 clocks a piece more (497 us); pieces loaded a step
// ahead into registers and a fifth buffer, before the values' buffers were given back
// early, 459 us for 457.
// Tensor memory: S_g at columns 128 g (P_g, fp16, over its first 64), O_g at
// 256 + 128 g.  MMA order of tile j: PV_0(j), S_0(j+1), PV_1(j), S_1(j+1); with one
// row block S of the tiles in turn in both places and S(j+1) before PV(j), so that
// a tile's softmax follows the one before without a pause (40 rows of 131072: 39 -> 34 us
// when it was built, 30 now).
// fp16 outputs: probabilities are rounded to fp16 before they meet the values
// (an output is off by 2.6e-4 of itself, 2-norm, 2.1e-4 of them the rounding of
// the output); fp32 outputs: two fp16 parts (22 bits), half as many products
// again (613 us for 428).  Their sum is taken before the rounding, in fp32.
// The key tiles of pair blocks that do not fill the GPU are split over CTAs
// (tile_split), whose unnormalised rows with their maximum and sum are joined
// by a second kernel.
// Every wait is bounded as in the prefill kernels (BGTQ_STATUS_TIMEOUT).
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "fp4.cuh"
#include "tc_common.cuh"

namespace bgtq {
namespace {

constexpr int kRows = 128;                      // rows of a block
constexpr int kKeys = 128;                      // positions of a tile
constexpr int kTileGroups = kKeys / kGroup;
constexpr int kTileThreads = 512;
constexpr int kDqWarp0 = 9, kDqWarps = 7;        // decoding warps
constexpr uint32_t kHalfBytes = kGroupBytes / 2;  // a group's keys or values: codes, then scales
constexpr int kRingHalves = 4;                    // of them of a decoding warp in shared memory
static_assert(kDqWarps <= kTileGroups, "a decoding warp has a piece in every tile (of eight or sixteen)");
constexpr uint32_t kTile = kRows * kD * 2;      // one 128 x 128 fp16 tile
constexpr uint32_t kBox = kTile / 2;            // 64 columns of it (128 rows x 128 B)
constexpr uint32_t kOffQ = 0, kOffK = 2 * kTile, kOffV = 4 * kTile, kOffStage = 6 * kTile;
constexpr uint32_t kTilesSmem = kOffStage + kDqWarps * kRingHalves * kHalfBytes + 1024;
constexpr uint32_t kTmemCols = 512;
// a row's reference stays kLift below its largest logit when set and moves when
// a logit passes it by kLift + kHeadroom: P up to 2^15, its small ones above
// fp16's smallest numbers
constexpr float kLift = 7.0f, kHeadroom = 8.0f, kLow = -1.0e30f;
// registers: what the block is launched with (128 x 512) shared out anew; the
// launcher checks the sum (more would be waited for without end)
constexpr int kSoftmaxRegs = 184, kOtherRegs = 72;

enum {
    kBarQ = 0,
    kBarKFull = 2,
    kBarVFull = 4,
    kBarKEmpty = 6,
    kBarVEmpty = 8,
    kBarS = 10,
    kBarP = 12,
    kBarO = 14,
    kBarDrain = 16,
    kNumBars
};

struct TileParams {
    RopeParams rope;
    RowsView q;
    Fp4Map map;
    const int32_t* seq_lens;
    int64_t max_len;
    int batch, t, group, H;
    int heads;        // batch * H
    int blocks;       // pairs of row blocks of a KV head
    int n_whole;      // units (pair block, head) whose tiles one CTA takes; they come first
    int n_split;      // the other units: each in `parts` splits of part_tiles tiles (the last: what is left)
    int parts, part_tiles;
    void* out;
    int out_dtype;
    float scale_log2;
    float* part_o;    // [parts][n_split][256][128]
    float2* part_ml;  // [parts][n_split][256]
    int32_t* status;
};

// Tiles that the rows of pair block pb see, for a sequence of n tokens.
__device__ __forceinline__ int block_tiles(const TileParams& p, int pb, int n) {
    const int last = min(p.t * p.group, (pb + 1) * 2 * kRows) - 1;
    return (max(0, n - p.t + 1 + last / p.group) + kKeys - 1) / kKeys;
}
__device__ __forceinline__ int clamp_len(const TileParams& p, int b) {
    const int64_t n = p.seq_lens[b];
    return n < 0 ? 0 : n > p.max_len ? (int)p.max_len : (int)n;
}

bool descriptors_valid() {
    if (!instr_desc_ok(instr_desc(kRows, kKeys, 0), 0)) return false;
    constexpr uint32_t kMaxSmem = 227u * 1024u;
    for (uint32_t base = 0; base + kTilesSmem <= kMaxSmem + 1024; base += 1024)
        for (int k = 0; k < 8; ++k)
            for (uint32_t tile = 0; tile < 6; ++tile)
                if (!smem_desc_ok(base + tile * kTile + (uint32_t)(k >> 2) * kBox + (uint32_t)(k & 3) * 32, 16, 1024)) return false;
    return true;
}

// Byte of element (row, col) of a tile: 64-column boxes, 16-byte pieces of a row exchanged by its low bits.
__device__ __forceinline__ uint32_t tile_at(int row, int col) {
    return (uint32_t)(col >> 6) * kBox + (uint32_t)row * 128u + ((((uint32_t)col >> 3) & 7u) ^ ((uint32_t)row & 7u)) * 16u +
           ((uint32_t)col & 7u) * 2u;
}
__device__ __forceinline__ void st_shared_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Writes of this thread become visible to the tensor cores (asynchronous proxy).
__device__ __forceinline__ void fence_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ uint32_t u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// What a lane's place in a warp says about where it reads and writes.
struct Place {
    uint32_t k_in, ks_in, k_out[4];  // keys: offsets of its codes and scales in a piece, of its stores in a group's rows
    uint32_t v_in, vs_in, v_out;     // values likewise; v_out without the group's columns
    uint32_t g16;                    // (lane / 4) * 16
    __device__ __forceinline__ explicit Place(int lane) {
        // Keys: a lane takes 4 dims of every block of a position, two positions in
        // turn.  The positions of 8 lanes are an even and an odd one, those of 16
        // lanes differ in bits 1-2, so that loads and stores fall on distinct banks.
        const int i = lane >> 2, c = lane & 3;
        const int pos = i < 4 ? (i << 1) + (i & 1) : ((i - 4) << 1) + 1 - (i & 1);  // 0 3 4 7 1 2 5 6
        k_in = 64 * pos + 16 * c;
        ks_in = 8 * pos;
#pragma unroll
        for (int j = 0; j < 4; ++j) k_out[j] = 128u * pos + 8u * (c & 1) + 16u * ((uint32_t)(2 * j + (c >> 1)) ^ (uint32_t)pos);
        v_in = 16 * lane;
        vs_in = 32 * c;
        v_out = 128u * i + 4u * c;
        g16 = 16u * i;
    }
};

template <int kAt>
__device__ __forceinline__ void store2(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.b32 [%0 + %3], {%1, %2};" ::"r"(a), "r"(x), "r"(y), "n"(kAt) : "memory");
}
template <int kAt>
__device__ __forceinline__ void store1(uint32_t a, uint32_t x) {
    asm volatile("st.shared.b32 [%0 + %2], %1;" ::"r"(a), "r"(x), "n"(kAt) : "memory");
}

// Blocks 2 kJJ and 2 kJJ + 1 of a position's keys (row 8 kIt + .. of the piece's rows).
template <int kIt, int kJJ>
__device__ __forceinline__ void key_blocks(uint32_t w, uint32_t sw, const uint32_t (&out)[4]) {
    const __half2 s = fp4_scales<(kJJ & 1) * 2>(sw), s0 = __low2half2(s), s1 = __high2half2(s);
    __half2 x[4];
    fp4_numbers(w, x);
    constexpr int kAt = kIt * 1024 + (kJJ >> 1) * (int)kBox;
    store2<kAt>(out[(2 * kJJ) & 3], u32(__hmul2(x[0], s0)), u32(__hmul2(x[1], s0)));
    store2<kAt>(out[(2 * kJJ + 1) & 3], u32(__hmul2(x[2], s1)), u32(__hmul2(x[3], s1)));
}

template <int kIt>
__device__ __forceinline__ void key_row(const uint4& w, const uint32_t (&s)[2], const uint32_t (&out)[4]) {
    key_blocks<kIt, 0>(w.x, s[0], out);
    key_blocks<kIt, 1>(w.y, s[0], out);
    key_blocks<kIt, 2>(w.z, s[1], out);
    key_blocks<kIt, 3>(w.w, s[1], out);
}

// Keys of groups kPer pr .. of a tile.
template <int kPer>
__device__ __forceinline__ void decode_keys(const Place& at, uint32_t img, uint32_t tile, int pr) {
    uint4 w[2 * kPer];
    uint32_t s[2 * kPer][2];
#pragma unroll
    for (int it = 0; it < 2 * kPer; ++it) {
        w[it] = ld_shared_v4(img + at.k_in + 512 * it);
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                     : "=r"(s[it][0]), "=r"(s[it][1])
                     : "r"(img + kPer * kGroupV + at.ks_in + 64 * it)
                     : "memory");
    }
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = tile + 2048u * kPer * pr + at.k_out[j];
    key_row<0>(w[0], s[0], out);
    key_row<1>(w[1], s[1], out);
    if constexpr (kPer == 2) {
        key_row<2>(w[2], s[2], out);
        key_row<3>(w[3], s[3], out);
    }
}

// Block kJ (dims 16 kJ ..) of the values of four positions.
template <int kJ>
__device__ __forceinline__ void value_block(uint32_t w, uint32_t sw, uint32_t a0, uint32_t a1) {
    const __half2 f0 = fp4_scales<0>(sw), f1 = fp4_scales<2>(sw);
    __half2 x[4];
    fp4_numbers(w, x);
    store1<2048 * kJ>(a0, u32(__hmul2(x[0], f0)));
    store1<2048 * kJ + 1024>(a0, u32(__hmul2(x[1], f0)));
    store1<2048 * kJ>(a1, u32(__hmul2(x[2], f1)));
    store1<2048 * kJ + 1024>(a1, u32(__hmul2(x[3], f1)));
}

// Values of groups kPer pr .., transposed; `live`: positions from the first
// group's on that exist (the others become zeros, whatever their bytes).
template <int kPer>
__device__ __forceinline__ void decode_values(const Place& at, uint32_t img, uint32_t tile, int pr, int live, int lane) {
    uint4 w[2 * kPer], s[2 * kPer];
#pragma unroll
    for (int i = 0; i < 2 * kPer; ++i) {
        w[i] = ld_shared_v4(img + at.v_in + 512 * i);
        s[i] = ld_shared_v4(img + kPer * kGroupV + at.vs_in + 128 * (i >> 1) + 16 * (i & 1));
    }
    if (live < kPer * kGroup) {
#pragma unroll
        for (int i = 0; i < 2 * kPer; ++i) {
            uint32_t keep = 0xffffffffu;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (kGroup * (i >> 1) + 2 * (lane & 3) + (e & 1) + 8 * (e >> 1) >= live) keep &= ~(0xffu << (8 * e));
            s[i].x &= keep, s[i].y &= keep, s[i].z &= keep, s[i].w &= keep;
        }
    }
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
        // positions 16 gr + 2 c (+ 1) and + 8: columns of the transposed tile
        const int gr = kPer * pr + x;
        const uint32_t box = tile + (uint32_t)(gr >> 2) * kBox + at.v_out;
        const uint32_t a0 = box + ((uint32_t)(32 * (gr & 3)) ^ at.g16), a1 = box + ((uint32_t)(32 * (gr & 3) + 16) ^ at.g16);
        const uint4 &w0 = w[2 * x], &w1 = w[2 * x + 1], &s0 = s[2 * x], &s1 = s[2 * x + 1];
        value_block<0>(w0.x, s0.x, a0, a1);
        value_block<1>(w0.y, s0.y, a0, a1);
        value_block<2>(w0.z, s0.z, a0, a1);
        value_block<3>(w0.w, s0.w, a0, a1);
        value_block<4>(w1.x, s1.x, a0, a1);
        value_block<5>(w1.y, s1.y, a0, a1);
        value_block<6>(w1.z, s1.z, a0, a1);
        value_block<7>(w1.w, s1.w, a0, a1);
    }
}

__device__ __forceinline__ void store_row(const TileParams& p, int b, int h, int r, const float* o, int col, float f) {
    const int i = r / p.group, a = r - i * p.group;
    const int64_t at = (((int64_t)b * p.H * p.group + h * p.group + a) * p.t + i) * kD + col;
    if (p.out_dtype) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
#pragma unroll
        for (int k = 0; k < 8; ++k) dst[k] = make_float4(o[4 * k] * f, o[4 * k + 1] * f, o[4 * k + 2] * f, o[4 * k + 3] * f);
    } else {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__half*>(p.out) + at);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            dst[k] = make_uint4(pack_h2(o[8 * k] * f, o[8 * k + 1] * f), pack_h2(o[8 * k + 2] * f, o[8 * k + 3] * f),
                                pack_h2(o[8 * k + 4] * f, o[8 * k + 5] * f), pack_h2(o[8 * k + 6] * f, o[8 * k + 7] * f));
    }
}

// The thread's query row (r of the head's packed rows) into row `at` of a tile
// at `tile`, rotated; returns the last position that it sees (-1: none).
__device__ __forceinline__ int bring_query(const TileParams& p, uint32_t tile, int at, int b, int h, int r, int n) {
    int lim = -1;
    int pos[kMaxAxes];
    const __half* row = nullptr;
    if (r < p.t * p.group) {
        const int i = r / p.group, a = r - i * p.group;
        lim = n - p.t + i;
        if (lim >= 0) {
            row = static_cast<const __half*>(p.q.p) + b * p.q.sb + (int64_t)(h * p.group + a) * p.q.sh + i * p.q.st;
            if (p.rope.cos && !rope_positions(p.rope, (int64_t)b * p.t + i, lim, pos)) {
                if (p.status) atomicOr(p.status, BGTQ_STATUS_ROPE_RANGE);
                row = nullptr;
                lim = -1;
            }
        } else {
            lim = -1;
        }
    }
    const bool split = p.rope.cos == nullptr || p.rope.layout == 0;
#pragma unroll 2
    for (int m = 0; m < 8; ++m) {
        const int da = split ? 8 * m : 16 * m, db = split ? 64 + 8 * m : 16 * m + 8;
        uint32_t x[4] = {0u, 0u, 0u, 0u}, y[4] = {0u, 0u, 0u, 0u};
        if (row) {
            const uint4 u = *reinterpret_cast<const uint4*>(row + da), v = *reinterpret_cast<const uint4*>(row + db);
            x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
            y[0] = v.x, y[1] = v.y, y[2] = v.z, y[3] = v.w;
            if (p.rope.cos) rope_rotate8(p.rope, pos, 8 * m, x, y);
        }
        st_shared_v4(tile + tile_at(at, da), x[0], x[1], x[2], x[3]);
        st_shared_v4(tile + tile_at(at, db), y[0], y[1], y[2], y[3]);
    }
    return lim;
}

template <bool kTwo, int kPer>
__global__ void __launch_bounds__(kTileThreads, 1) fp4_tiles_kernel(const __grid_constant__ TileParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_bar[kNumBars];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // units with the most tiles (a head's last rows) first; of split units all first parts, then all second ones
    int unit = blockIdx.x, part = 0;
    const bool cut = unit >= p.n_whole;
    if (cut) {
        part = (unit - p.n_whole) / p.n_split;
        unit -= part * p.n_split;
    }
    const int pb = p.blocks - 1 - unit / p.heads, head = unit % p.heads;
    const int b = head / p.H, h = head - b * p.H;
    const int rows = p.t * p.group;
    const int r0 = pb * 2 * kRows;
    const int ng = kPer == 1 && r0 + kRows < rows ? 2 : 1;  // (kPer = 2: up to kRows rows)
    const uint32_t bar0 = smem_u32(&s_bar[0]);
    volatile int* abort_flag = &s_abort;
#define BAR(i) (bar0 + 8u * (uint32_t)(i))
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n = clamp_len(p, b);
    if (tid == 0 && part == 0 && pb == 0 && h == 0 && p.status && n != p.seq_lens[b]) {
        atomicOr(p.status, BGTQ_STATUS_SEQLEN_CAPACITY);
        debug_in_range(false, p.status);  // groups past the bound
    }
    const int tiles = block_tiles(p, pb, n);
    const int j0 = part * p.part_tiles, j1 = cut ? min(tiles, j0 + p.part_tiles) : tiles;
    if (part > 0 && j0 >= tiles) return;
    const bool whole = j0 == 0 && j1 == tiles;  // this CTA has every position that its rows see
    const int nkt = max(0, j1 - j0);

    if (tid == 0) {
        s_abort = 0;
        auto lanes_of = [&](int g) { return max(1, min(kRows, (rows - r0 - kRows * g + 31) & ~31)); };  // of warps with a row
        for (int i = 0; i < kNumBars; ++i)
            mbar_init(BAR(i), i < kBarKFull ? 4 : i < kBarKEmpty ? kTileGroups / kPer : (i == kBarP || i == kBarP + 1) ? lanes_of(ng == 1 ? 0 : i - kBarP) : 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8 && nkt > 0) {
            // ---- MMA issue
            constexpr uint32_t id = instr_desc(kRows, kKeys, 0);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            auto wait = [&](int bar, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait(BAR(bar), parity & 1u, abort_flag, p.status));
            };
            auto step = [](int k) { return (uint32_t)(k >> 2) * kBox + (uint32_t)(k & 3) * 32u; };
            // S of row block g at tensor-memory column 128 to (one row block: its tiles in turn)
            auto issue_s = [&](int g, int to, int j) {
                const uint32_t qa = sbase + kOffQ + g * kTile, ka = sbase + kOffK + (j & 1) * kTile;
#pragma unroll
                for (int k = 0; k < kD / 16; ++k)
                    mma_ss_warp(tm + 128u * to, smem_desc(qa + step(k), 16, 1024), smem_desc(ka + step(k), 16, 1024), id, k > 0);
                mma_commit_warp(BAR(kBarS + to));
            };
            auto issue_pv = [&](int g, int from, int j) {
                const uint32_t va = sbase + kOffV + (j & 1) * kTile;
#pragma unroll(kTwo ? 4 : 8)  // (all 16 products in line cost the warp registers that it has not)
                for (int k = 0; k < kKeys / 16; ++k) {
                    mma_ts_warp(tm + 256u + 128u * g, tm + 128u * from + 8u * k, smem_desc(va + step(k), 16, 1024), id,
                                (j > 0 || k > 0) ? 1u : 0u);
                    if (kTwo) mma_ts_warp(tm + 256u + 128u * g, tm + 128u * from + 64u + 8u * k, smem_desc(va + step(k), 16, 1024), id, 1u);
                }
            };
            bool ok = wait(kBarQ, 0) && (ng < 2 || wait(kBarQ + 1, 0)) && wait(kBarKFull, 0);
            if (ok) {
                tc_fence_after();
                for (int g = 0; g < ng; ++g) issue_s(g, g, 0);
                mma_commit_warp(BAR(kBarKEmpty));
            }
            for (int j = 0; ok && j < nkt; ++j) {
                const int s = j & 1;
                const bool next = j + 1 < nkt;
                // (two blocks: both waits before the first product; with the keys' in front of
                // S_0 alone the blocks lose their turns, 461 us for 428)
                ok = (ng == 1 || wait(kBarVFull + s, (uint32_t)(j >> 1))) && (!next || wait(kBarKFull + (s ^ 1), (uint32_t)((j + 1) >> 1)));
                if (!ok) break;
                if (ng == 1) {
                    // one row block: the next tile's S while this one's softmax runs.  Buffers are
                    // given back in order, each after the ones before it have arrived: a wait for
                    // one is then never told from its barrier's phase before by time alone.
                    if (next) {
                        tc_fence_after();
                        issue_s(0, s ^ 1, j + 1);
                        if (!(ok = (j == 0 || wait(kBarVEmpty + (s ^ 1), (uint32_t)((j - 1) >> 1))) && wait(kBarKEmpty + s, (uint32_t)(j >> 1)))) break;
                        mma_commit_warp(BAR(kBarKEmpty + (s ^ 1)));
                    }
                    if (!(ok = wait(kBarP + s, (uint32_t)(j >> 1)) && wait(kBarVFull + s, (uint32_t)(j >> 1)))) break;
                    tc_fence_after();
                    issue_pv(0, s, j);
                    mma_commit_warp(BAR(kBarVEmpty + s));
                    if (!next) mma_commit_warp(BAR(kBarO));
                    continue;
                }
                for (int g = 0; g < 2 && ok; ++g) {
                    if (!(ok = wait(kBarP + g, (uint32_t)j))) break;
                    tc_fence_after();
                    issue_pv(g, g, j);
                    // (a commit covers what was issued before it: the values' before S_1, 457 -> 430 us)
                    if (g == 1) mma_commit_warp(BAR(kBarVEmpty + s));
                    if (next) {
                        issue_s(g, g, j + 1);
                    } else {
                        mma_commit_warp(BAR(kBarO + g));
                    }
                }
                if (ok && next) mma_commit_warp(BAR(kBarKEmpty + (s ^ 1)));
            }
            // every MMA issued has completed before the CTA ends
            mma_commit_warp(BAR(kBarDrain));
            mbar_wait(BAR(kBarDrain), 0, abort_flag, p.status, false);
        } else if (warp >= kDqWarp0) {
            // ---- decoding: a tile's pieces are the keys, then the values of kPer groups
            // each; a warp takes every kDqWarps-th, the next kRing of them on their way
            constexpr int kPieces = kTileGroups / kPer, kRing = kRingHalves / kPer;
            constexpr uint32_t kPieceScales = kPer * kGroupV, kPieceBytes = kPer * kHalfBytes;
            const int w = warp - kDqWarp0;
            const int n_groups = (n + kGroup - 1) / kGroup, first = j0 * kTileGroups;
            const int count = max(0, min(kTileGroups * nkt, n_groups - first));  // groups of the CTA's tiles
            const Place at(lane);
            const uint32_t ring = sbase + kOffStage + w * (kRing * kPieceBytes);
            const bool paged = p.map.page_table != nullptr;
            const uint8_t* flat = paged ? nullptr : p.map.group(b, h, first);
            auto group = [&](int x) -> const uint8_t* {
                if (!paged) return flat + (int64_t)x * kGroupBytes;
                const uint8_t* src = p.map.group(b, h, first + x);
                if (src) return src;
                if (lane == 0 && p.status) atomicOr(p.status, BGTQ_STATUS_PAGE_RANGE);
                return p.map.base;  // (some group of the pool: the output is unspecified)
            };
            auto fetch = [&](int u, int st) {
                const int x = u / (2 * kPieces) * kTileGroups + kPer * (u % kPieces);
                if (x < count) {
                    const bool two = kPer == 2 && x + 1 < count, values = u & kPieces;
                    const uint8_t* src = group(x);
                    const uint8_t* next = !two ? src : !paged || p.map.lg > 0 ? src + kGroupBytes : group(x + 1);
                    const uint32_t dst = ring + st * kPieceBytes + 16 * lane, codes = 16 * lane + (values ? kGroupV : 0);
                    copy16(dst, src + codes);
                    copy16(dst + 512, src + codes + 512);
                    if (two) {
                        copy16(dst + 1024, next + codes);
                        copy16(dst + 1536, next + codes + 512);
                    }
                    if (lane < 8 * kPer)
                        copy16(dst + kPieceScales, (lane < 8 ? src : next) + (values ? kGroupVs : kGroupKs) + 16 * (lane & 7));
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait(bar, parity & 1u, abort_flag, p.status));
            };
            for (int i = 0; i < kRing; ++i) fetch(w + i * kDqWarps, i);
            int st = 0;
            for (int u = w; u < 2 * kPieces * nkt; u += kDqWarps) {
                const int j = u / (2 * kPieces), pr = u % kPieces, s = j & 1, x = kTileGroups * j + kPer * pr;
                const uint32_t img = ring + st * kPieceBytes;
                const bool keys = !(u & kPieces);
                // the tile's buffer is free, the piece has landed.  (The wait could be mistaken for
                // that of tile j - 4 while its buffer is out.  With pieces of one group this warp
                // waited for it itself, tile by tile; with two it may have had none of this kind,
                // but waited for one that was given back after it, see the MMA warp.)
                if (j >= 2 && !wait(BAR((keys ? kBarKEmpty : kBarVEmpty) + s), (uint32_t)((j >> 1) - 1))) break;
                asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
                __syncwarp();
                if (keys)
                    decode_keys<kPer>(at, img, sbase + kOffK + s * kTile, pr);
                else
                    decode_values<kPer>(at, img, sbase + kOffV + s * kTile, pr, n - (first + x) * kGroup, lane);
                fence_to_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR((keys ? kBarKFull : kBarVFull) + s));
                fetch(u + kRing * kDqWarps, st);
                if (++st == kRing) st = 0;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
        __syncwarp();
    } else {
        // ---- softmax warpgroups
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int g = warp >> 2;
        const int r = r0 + kRows * g + 32 * (warp & 3) + lane;  // packed row = tensor-memory lane
        if (g < ng) {
            const int lim = bring_query(p, sbase + kOffQ + g * kTile, 32 * (warp & 3) + lane, b, h, r, n);
            fence_to_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(kBarQ + g));
            const int lim_min = __reduce_min_sync(0xffffffffu, r < rows ? lim : n - 1);
            const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
            const uint32_t tO = tmem + lanes + 256u + 128u * g;
            const float c = p.scale_log2;
            float m = kLow, l = 0.0f;
            bool ok = true;
            // (a warp without a row leaves its lanes' P and O as they are)
            const int n_soft = __shfl_sync(0xffffffffu, r < rows ? nkt : 0, 0);
            for (int j = 0; j < n_soft; ++j) {
                const int at = ng == 1 ? j & 1 : g;  // its S
                const uint32_t tS = tmem + lanes + 128u * at;
                if (!__all_sync(0xffffffffu, mbar_wait(BAR(kBarS + at), (ng == 1 ? j >> 1 : j) & 1, abort_flag, p.status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                float s[kKeys];
#pragma unroll
                for (int q = 0; q < kKeys / 32; ++q) tmem_ld32(tS + 32 * q, s + 32 * q);
#pragma unroll
                for (int q = 0; q < kKeys / 32; ++q) tmem_wait_ld32(s + 32 * q);
                const int k0 = (j0 + j) * kKeys;
                if (k0 + kKeys - 1 > lim_min) {
                    const int last = lim - k0;
#pragma unroll
                    for (int k = 0; k < kKeys; ++k)
                        if (k > last) s[k] = -INFINITY;
                }
                float mx[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) mx[i] = s[i];
#pragma unroll
                for (int k = 8; k < kKeys; ++k) mx[k & 7] = fmaxf(mx[k & 7], s[k]);
                const float mt = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                       fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * c;
                float f = 1.0f;
                const bool raise = mt > m + (kLift + kHeadroom);
                if (raise) {
                    f = ex2(m - (mt - kLift));  // (0 from "no position yet")
                    m = mt - kLift;
                    l *= f;
                }
                if (j > 0 && __any_sync(0xffffffffu, raise)) {
                    // the row's O so far is in tensor memory; PV of tile j - 1 has
                    // completed (two blocks: S of tile j was issued after it; one: its values are given back)
                    if (ng == 1 && !__all_sync(0xffffffffu, mbar_wait(BAR(kBarVEmpty + ((j - 1) & 1)), ((j - 1) >> 1) & 1, abort_flag, p.status))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int q = 0; q < kD / 32; ++q) {
                        float o[32];
                        tmem_ld32(tO + 32 * q, o);
                        tmem_wait_ld32(o);
                        uint32_t w[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(o[i] * f);
                        tmem_st32(tO + 32 * q, w);
                    }
                }
                const uint64_t c2 = pack2(c, c), m2 = pack2(-m, -m);
                uint64_t l2[4];
                // P over the first 64 columns of S (already read); its second part over the others
                if constexpr (kTwo) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const int i = 16 * q + x;
                            const uint64_t e = exp2_pair(fma2(pack2(s[2 * i], s[2 * i + 1]), c2, m2));
                            l2[i & 3] = i < 4 ? e : add2(l2[i & 3], e);
                            const float2 w = unpack2(e);
                            const __half2 hh = __floats2half2_rn(w.x, w.y);
                            const float2 back = __half22float2(hh);
                            hi[x] = u32(hh);
                            lo[x] = pack_h2(w.x - back.x, w.y - back.y);
                        }
                        tmem_st16(tS + 16 * q, hi);
                        tmem_st16(tS + 64 + 16 * q, lo);
                    }
                } else {
                    uint32_t pk[kKeys / 2];
#pragma unroll
                    for (int i = 0; i < kKeys / 2; ++i) {
                        const uint64_t e = exp2_pair(fma2(pack2(s[2 * i], s[2 * i + 1]), c2, m2));
                        l2[i & 3] = i < 4 ? e : add2(l2[i & 3], e);
                        const float2 w = unpack2(e);
                        pk[i] = pack_h2(w.x, w.y);
                    }
                    tmem_st32(tS, pk);
                    tmem_st32(tS + 32, pk + 32);
                }
                const float2 a = unpack2(add2(l2[0], l2[1])), b2 = unpack2(add2(l2[2], l2[3]));
                l += (a.x + a.y) + (b2.x + b2.y);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(BAR(kBarP + at));
            }
            if (nkt > 0) ok = ok && __all_sync(0xffffffffu, mbar_wait(BAR(kBarO + g), 0, abort_flag, p.status));
            if (ok) {
                tc_fence_after();
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                const int64_t at = ((int64_t)part * p.n_split + (unit - p.n_whole)) * (2 * kRows) + (r - r0);
                if (!whole && r < rows) p.part_ml[at] = make_float2(m, l);
#pragma unroll 1
                for (int q = 0; q < kD / 32; ++q) {
                    float o[32];
                    if (nkt > 0) {
                        tmem_ld32(tO + 32 * q, o);
                        tmem_wait_ld32(o);
                    }
                    // a row that saw nothing: zeros, whatever its accumulator holds
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = nkt > 0 && (l > 0.0f || l != l) ? o[i] : 0.0f;
                    if (r >= rows) continue;
                    if (whole) {
                        store_row(p, b, h, r, o, 32 * q, l != l ? l : inv);
                    } else {
                        float4* dst = reinterpret_cast<float4*>(p.part_o + at * kD + 32 * q);
#pragma unroll
                        for (int k = 0; k < 8; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
#undef BAR
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    }
}

// Joins the splits' rows: kWide, many splits: a block of eight warps a row, a
// warp every eighth split; else a warp a row.  Four dims a lane.
template <bool kWide>
__global__ void __launch_bounds__(256) fp4_join_kernel(const __grid_constant__ TileParams p) {
    __shared__ __align__(16) float s_o[8][kD];
    __shared__ float2 s_ml[8];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t total = (int64_t)p.n_split * (2 * kRows);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t slot_row = kWide ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 8 + warp;
    const int unit = p.n_whole + (int)(slot_row / (2 * kRows));
    const int pb = p.blocks - 1 - unit / p.heads, head = unit % p.heads;
    const int r = pb * 2 * kRows + (int)(slot_row % (2 * kRows));
    if (r >= p.t * p.group) return;
    const int b = head / p.H, h = head - b * p.H;
    const int tiles = block_tiles(p, pb, clamp_len(p, b));
    const int active = (tiles + p.part_tiles - 1) / p.part_tiles;
    if (active <= 1) return;  // (written by its CTA)
    constexpr int kStep = kWide ? 8 : 1, kAhead = kWide ? 8 : 4;
    float m = kLow, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int x0 = kWide ? warp : 0; x0 < active; x0 += kStep * kAhead) {
        float2 ml[kAhead];
        float4 v[kAhead];
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            const int x = x0 + kStep * y;
            ml[y] = make_float2(kLow, 0.0f);
            v[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (x < active) {
                ml[y] = p.part_ml[x * total + slot_row];
                v[y] = *reinterpret_cast<const float4*>(p.part_o + (x * total + slot_row) * kD + 4 * lane);
            }
        }
        float top = m;
#pragma unroll
        for (int y = 0; y < kAhead; ++y) top = fmaxf(top, ml[y].x);
        const float f0 = ex2(m - top);
        m = top;
        l *= f0;
        o.x *= f0, o.y *= f0, o.z *= f0, o.w *= f0;
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
            const float f = ex2(ml[y].x - m);
            l += f * ml[y].y;
            o.x += f * v[y].x, o.y += f * v[y].y, o.z += f * v[y].z, o.w += f * v[y].w;
        }
    }
    int d = 4 * lane;
    if constexpr (kWide) {
        // 16 dims a warp, a warp's partial for four lanes
        *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = o;
        if (lane == 0) s_ml[warp] = make_float2(m, l);
        __syncthreads();
        const int share = lane >> 2;
        d = 16 * warp + 4 * (lane & 3);
        const float2 ml = s_ml[share];
        o = *reinterpret_cast<const float4*>(&s_o[share][d]);
        m = ml.x;
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, y));
        const float f = ex2(ml.x - m);
        l = f * ml.y;
        o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) {
            l += __shfl_xor_sync(0xffffffffu, l, y);
            o.x += __shfl_xor_sync(0xffffffffu, o.x, y);
            o.y += __shfl_xor_sync(0xffffffffu, o.y, y);
            o.z += __shfl_xor_sync(0xffffffffu, o.z, y);
            o.w += __shfl_xor_sync(0xffffffffu, o.w, y);
        }
        if (share != 0) return;
    }
    const float inv = l > 0.0f ? 1.0f / l : l != l ? l : 0.0f;
    const int i = r / p.group, a = r - i * p.group;
    const int64_t at = (((int64_t)b * p.H * p.group + h * p.group + a) * p.t + i) * kD + d;
    if (p.out_dtype)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    else
        *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + at) =
            make_uint2(pack_h2(o.x * inv, o.y * inv), pack_h2(o.z * inv, o.w * inv));
}

constexpr int kSms = 152, kLeastTiles = 2;

// Units (pair blocks of all heads) onto the GPU's 152 SMs, one CTA each.  More
// units than SMs: whole ones for the full rounds, the rest split over the SMs.
// Fewer: p equal parts and one smaller one, of which an SM that has no large
// part takes k in turn while the large ones run: k s = m, p m + s = tiles
// (128 units of 272 tiles: 233 + 39).  Parts of kLeastTiles at least: a CTA's
// own start and end take as long as about three tiles, but CTAs of few units
// would be idle; a smaller part of eight at least.
struct TileSplit {
    int64_t n_whole, n_split;
    int parts, part_tiles;
};
TileSplit tile_split(int64_t units, int64_t max_len) {
    const int64_t tiles = std::max<int64_t>(1, (max_len + kKeys - 1) / kKeys), small = 8;
    const int64_t n_split = units % kSms, n_whole = units - n_split;
    if (n_split == 0 || tiles < 2 * kLeastTiles) return {units, 0, 1, (int)tiles};
    const int64_t p = kSms / n_split, free = kSms - p * n_split;
    int64_t m = (tiles + p - 1) / p;
    if (free > 0 && n_whole == 0) {
        const int64_t k = (n_split + free - 1) / free;
        const int64_t m2 = (k * tiles + p * k) / (p * k + 1);  // rounded up
        if (m2 + small < m && tiles - p * m2 >= small) m = m2;
    }
    m = std::max<int64_t>(m, kLeastTiles);
    const int64_t parts = (tiles + m - 1) / m;
    if (parts == 1) return {units, 0, 1, (int)tiles};
    return {n_whole, n_split, (int)parts, (int)m};
}

int64_t pair_blocks(int64_t rows) { return (rows + 2 * kRows - 1) / (2 * kRows); }

}  // namespace

// Room for the splits' rows of any shape up to this one: at most kSms of equal
// parts and kSms smaller ones, none of less than kLeastTiles but the last.
size_t fp4_tiles_workspace_bytes(int64_t heads, int64_t rows, int64_t max_len) {
    const int64_t tiles = std::max<int64_t>(1, (max_len + kKeys - 1) / kKeys);
    auto most = [](int64_t n) { return std::min<int64_t>(n, 2 * kSms); };  // (the product of the largest shapes passes 64 bits)
    const int64_t slots = most(most(heads) * most(pair_blocks(rows)) * most((tiles + kLeastTiles - 1) / kLeastTiles));
    return (size_t)slots * 2 * kRows * (8 + 4 * kD);
}

cudaError_t launch_fp4_tiles(cudaStream_t s, const Fp4Attn& a, void* ws) {
    static std::mutex mu;
    static bool done[64] = {false};
    static const bool desc_ok = descriptors_valid();
    if (!desc_ok) return cudaErrorInvalidValue;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!done[dev]) {
            for (auto kernel : {fp4_tiles_kernel<false, 1>, fp4_tiles_kernel<false, 2>, fp4_tiles_kernel<true, 1>}) {
                cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTilesSmem);
                cudaFuncAttributes fa;
                if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kernel);
                if (e != cudaSuccess) return e;
                if (2 * kSoftmaxRegs + 2 * kOtherRegs > 4 * fa.numRegs) return cudaErrorInvalidConfiguration;
            }
            done[dev] = true;
        }
    }
    const int64_t rows = (int64_t)a.t * a.group, heads = (int64_t)a.batch * a.map.H;
    TileParams p;
    p.rope = a.rope;
    p.q = a.q;
    p.map = a.map;
    p.seq_lens = a.seq_lens;
    p.max_len = std::min(a.max_len, a.cap);
    p.batch = a.batch;
    p.t = a.t;
    p.group = a.group;
    p.H = a.map.H;
    p.blocks = (int)pair_blocks(rows);
    const TileSplit sp = tile_split(heads * p.blocks, p.max_len);
    p.heads = (int)heads;
    p.n_whole = (int)sp.n_whole;
    p.n_split = (int)sp.n_split;
    p.parts = sp.parts;
    p.part_tiles = sp.part_tiles;
    p.out = a.out;
    p.out_dtype = a.out_dtype;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.part_o = static_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + (size_t)sp.parts * sp.n_split * 2 * kRows * kD * 4);
    p.status = a.status;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sp.n_whole + sp.n_split * sp.parts), 1, 1);
    cfg.blockDim = dim3(kTileThreads, 1, 1);
    cfg.dynamicSmemBytes = kTilesSmem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    // one row block, one part of P: pieces of two groups (32 x 8 heads of 8192, 64 rows a
    // head: 173 us, of one 199); else their bursts hold up the softmax (256 rows of 131072
    // in fp32 64 us, of one 53)
    cudaError_t e = cudaLaunchKernelEx(&cfg,
                                       a.out_dtype     ? fp4_tiles_kernel<true, 1>
                                       : rows <= kRows ? fp4_tiles_kernel<false, 2>
                                                       : fp4_tiles_kernel<false, 1>,
                                       p);
    if (e != cudaSuccess || sp.n_split == 0) return e;
    // a block a row while the rows alone do not fill the GPU (256 rows of 16 parts:
    // 12.7 us in all against 14.7; 2048 rows of 8: 27 against 20)
    const bool wide = sp.parts >= 8 && sp.n_split * 2 * kRows <= 8 * kSms;
    cfg.gridDim = dim3((unsigned)(sp.n_split * 2 * kRows / (wide ? 1 : 8)), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, wide ? fp4_join_kernel<true> : fp4_join_kernel<false>, p);
}

}  // namespace bgtq
