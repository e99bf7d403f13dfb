// Accumulated attention weights of a prompt's rows: for every key j of a KV
// head, the sum over the head's query heads and the rows i >= row0 of
//   exp(scale q_i . k_j - lse_i),   j <= i and (j < sinks or j > i - window),
// from the rows' log-sum-exp (bgtq_prefill_window_attn writes it).  These are
// the scores that rank the positions of a cache before it is cut to a budget.
//
// One pass over the (row, key) pairs, no softmax statistics to find: S^T =
// K_tile Q_tile^T on the tensor cores (tcgen05, 128 keys in the tensor-memory
// lanes, rows in the columns), so that a thread owns a key and its sum stays
// in a register over all rows: no reduction between threads, no atomics.  Per
// 128 x 256 pairs the MMAs take 1024 clocks, and so do the exponentials (32 a
// clock).  The MMAs read both operands from shared memory and use its whole
// bandwidth; reading a row's log-sum-exp from there for every product took as
// long again (183 us against 119 without those reads, 8191 rows x 16 query
// heads).  So -lse / scale rides in the product: a ninth step of 16 in K, the
// key side (256, 1, 1/256, 0 ..), the row side the three fp16 parts of
// -lse / scale that these factors join to fp32 accuracy.
//
// Persistent CTAs, one per SM, 18 warps:
//   warps 0-15   four warpgroups, thread = key = tensor-memory lane
//   warp 16      issues the MMAs (an elected lane) and owns the tensor memory
//   warp 17      issues the TMA copies (one thread)
// prefill_score_kernel (any number of rows): two key tiles stay, the row
// tiles (128 rows) of their query heads stream past them, so that a row tile
// is read from the L2 once per 256 keys (once per 128 would take the whole 64
// bytes a clock that an SM gets).  Accumulator 2 b + j: key tile j, row tiles
// of parity b, summed by warpgroup 2 b + j; the MMAs of the two key tiles
// alternate, because one 128-column accumulation after another leaves the
// tensor cores waiting for its result.  A tile's MMAs read 144 KB of shared
// memory and its copy writes 32 KB (1400 clocks at 128 bytes a clock, about
// what bounds it), a tile takes 1890 clocks: 1150 of MMAs at the tensor
// cores' rate, the rest the latency of the three waits before them.  (Those
// waits between the previous tile's MMAs, a second MMA warp, 256-column
// accumulators of one key tile and two CTAs per SM were all slower: 130, 151,
// 133 and 125 us against 125 for 8191 rows x 16 query heads.)  An item is a pair of key tiles and a
// share of the query heads; the key tiles are taken from the first on (the
// ones with the most rows), in a snake over the CTAs.  Where the query heads
// are shared out over several items a second kernel adds the sums, in order.
// prefill_score_rows_kernel (the rows of all the query heads of a KV head fit
// 256 columns, as the last 64 rows of 4 heads do): the rows stay, the key
// tiles stream, each read once from HBM; an accumulator of 256 columns is
// summed by two warpgroups.
// Rows that do not count get a weight exponent of -inf with their lse.  Where
// few rows count, a tile holds the rows of several query heads.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "tc_common.cuh"

namespace bgtq {
namespace {

constexpr int kPsKeys = 128, kPsCols = 128;                  // keys of a tile, rows of a row tile
constexpr int kPsGroups = 4;                                 // warpgroups
constexpr int kPsThreads = kPsGroups * 128 + 64;
constexpr int kPsMmaWarp = 4 * kPsGroups, kPsTmaWarp = kPsMmaWarp + 1;
constexpr int kPsStages = 3;                                 // row tiles in shared memory
constexpr uint32_t kPsTile = kPsKeys * kD * 2, kPsBox = kPsTile / 2;  // a tile of 128 keys or rows, a 64-column box of it
// two key tiles, the row tiles, and the boxes of the ninth step (its 16
// columns of a 64-column box): the keys', the rows' of either parity
constexpr uint32_t kPsOffRow = 2 * kPsTile, kPsOffKeyExt = kPsOffRow + kPsStages * kPsTile, kPsOffRowExt = kPsOffKeyExt + kPsBox;
constexpr uint32_t kPsSmem = kPsOffRowExt + 2 * kPsBox + 1024;  // (+ room to align the base to 1 KB)

enum {
    kPsBarK = 0,
    kPsBarKEmpty = 1,
    kPsBarQ = 2,
    kPsBarQEmpty = 5,
    kPsBarS = 8,
    kPsBarFree = 10,
    kPsBarExt = 12,
    kPsBarDrain = 14,
    kPsNumBars = 15
};

struct PsParams {
    const float* lse;  // [B][H*G][T]
    float* out;        // [B][H][stride], or [B][H][parts][T] for the join
    int64_t stride;
    int T, H, G, row0, sinks, window;
    int box;           // rows of a query head in a tile: all of them, or fewer with several heads in it
    int parts, heads;  // items per pair of key tiles, query heads of each
    int64_t items;
    float scale_log2;
    float unit_hi, unit_lo;  // 1 / scale
    int32_t* status;
};

// A row's log-sum-exp; -inf for a row that does not count.
__device__ __forceinline__ float row_lse(const PsParams& p, const float* lse_row, int row, bool counts) {
    return counts && row < p.T ? __ldg(lse_row + row) : -INFINITY;
}
// The ninth step's row side: -lse / scale as 256 a + b + c / 256 with fp16 a,
// b, c (33 bits; the quotient as the product with 1 / scale and its rounding
// error); a = -inf (a weight of 0) for a row that does not count or saw
// nothing, NaN where |lse / scale| is past the range of a.
__device__ __forceinline__ uint4 row_ext(const PsParams& p, float x) {
    if (!(fabsf(x) < INFINITY)) return make_uint4(x == x ? 0xFC00u : 0x7E00u, 0u, 0u, 0u);  // (a NaN stays one)
    const float n = -x * p.unit_hi, e = fmaf(-x, p.unit_lo, fmaf(-x, p.unit_hi, -n));
    if (fabsf(n) > 256.0f * 65504.0f) return make_uint4(0x7E00u, 0u, 0u, 0u);
    const __half a = __float2half_rn(n * (1.0f / 256.0f));
    const float r1 = fmaf(-256.0f, __half2float(a), n);  // exact
    const __half b = __float2half_rn(r1);
    const __half c = __float2half_rn(((r1 - __half2float(b)) + e) * 256.0f);
    return make_uint4((uint32_t)__half_as_ushort(a) | ((uint32_t)__half_as_ushort(b) << 16), (uint32_t)__half_as_ushort(c), 0u, 0u);
}

// Line `line` of a ninth step's box: 16 columns, the first eight `v`, the
// others 0, in the 128-byte swizzle (16-byte piece c of a line lies at piece
// c ^ (line mod 8)).
__device__ __forceinline__ void store_ext(uint32_t box, int line, uint4 v) {
    const uint32_t at = box + (uint32_t)line * 128u, sw = (uint32_t)(line & 7);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + 16u * sw), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + 16u * (1u ^ sw)), "r"(0u) : "memory");
}
// The keys' side, the same for every key: 256, 1, 1/256.
__device__ __forceinline__ void store_key_ext(uint32_t box, int line) {
    store_ext(box, line, make_uint4(0x5C00u | (0x3C00u << 16), 0x1C00u, 0u, 0u));
}
// Shared-memory writes before it are seen by MMAs issued after a barrier.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A tile of `cols` rows: row r of a 64-column box is its r-th 128-byte line;
// box rows of every head, in copies of at most 128 rows.
__device__ __forceinline__ void load_row_tile(const CUtensorMap* tq, uint32_t dst, const PsParams& p, int bh, int g_first,
                                              int n_heads, int head_tile, int row, int cols, uint32_t bar) {
    const uint32_t box_bytes = (uint32_t)cols * 128u;
    const int step = min(p.box, 128);
    for (int u = 0; u < cols / p.box; ++u) {
        // (past the last head: its rows again, not counted)
        const int g = g_first + min(head_tile * (cols / p.box) + u, n_heads - 1);
        for (int r = 0; r < p.box; r += step)
            for (int x = 0; x < 2; ++x)
                tma_load_3d(dst + x * box_bytes + (uint32_t)(u * p.box + r) * 128u, tq, 64 * x, row + r, bh * p.G + g, bar);
    }
}

// The row tiles of an item's 256 keys from k0: rows lo, lo + box, ... of each
// group of query heads.
struct RowTiles {
    int lo, n_rows_t, n;
    __device__ __forceinline__ RowTiles(const PsParams& p, int k0, int n_head_t) {
        lo = max(p.row0, k0);
        const int hi = p.sinks > k0 ? p.T : (int)min((int64_t)p.T, (int64_t)k0 + 2 * kPsKeys - 1 + p.window);
        n_rows_t = hi > lo ? (hi - lo + p.box - 1) / p.box : 0;
        n = n_rows_t * n_head_t;
    }
};

__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// This thread's sum over kCols columns from `taddr` of 2^(s c): the columns'
// weights for its key; kEdge: only the columns whose row within the box lies
// in [c_lo, c_hi) see the key.  The warp arrives once at `bar_free` when it
// has read the last of them.
template <int kCols, bool kEdge>
__device__ __forceinline__ float sum_columns(uint32_t taddr, uint64_t c2, int col0, int box_mask, int c_lo, int c_hi,
                                             uint32_t bar_free) {
    constexpr int kAcc = 4;
    uint64_t acc[kAcc];
#pragma unroll
    for (int q = 0; q < kCols / 32; ++q) {
        float s[32];
        tmem_ld32(taddr + 32 * q, s);
        tmem_wait_ld32(s);
        if (q == kCols / 32 - 1) {
            tc_fence_before();
            __syncwarp();
            if ((threadIdx.x & 31) == 0) mbar_arrive(bar_free);
        }
        if constexpr (kEdge) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int cc = (col0 + 32 * q + i) & box_mask;
                if (cc < c_lo || cc >= c_hi) s[i] = -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint64_t e = exp2_pair(mul2(pack2(s[2 * i], s[2 * i + 1]), c2));
            acc[i % kAcc] = q == 0 && i < kAcc ? e : add2(acc[i % kAcc], e);
        }
    }
    const float2 r = unpack2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])));
    return r.x + r.y;
}

// Item i of a CTA: rounds of gridDim.x items in alternating direction.
__device__ __forceinline__ int64_t snake(int64_t round) {
    const int64_t g = gridDim.x;
    return round * g + ((round & 1) ? g - 1 - blockIdx.x : blockIdx.x);
}

struct Item {
    int bh, part, k0, g_first, n_heads;
    __device__ __forceinline__ Item(const PsParams& p, int64_t i, int kv) {
        const int64_t per = (int64_t)kv * p.parts;
        const int r = (int)(i % per);
        k0 = (int)(i / per) * (2 * kPsKeys);
        bh = r / p.parts;
        part = r - bh * p.parts;
        g_first = part * p.heads;
        n_heads = min(p.heads, p.G - g_first);
    }
};

__global__ void __launch_bounds__(kPsThreads, 1)
    prefill_score_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk, PsParams p, int kv) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_bar[kPsNumBars];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ float s_half[2][2][kPsKeys];  // [key tile][item parity]: the sums of the odd row tiles
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u, srow = sbase + kPsOffRow;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per_tile = kPsCols / p.box;  // query heads of a tile
    const uint32_t bar0 = smem_u32(&s_bar[0]);
    volatile int* abort_flag = &s_abort;
#define BAR(i) (bar0 + 8u * (uint32_t)(i))

    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < kPsNumBars; ++i) mbar_init(BAR(i), (i == kPsBarFree || i == kPsBarFree + 1) ? 8 : (i == kPsBarExt || i == kPsBarExt + 1) ? 4 : 1);  // (warps)
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kPsMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(4 * kPsCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid < kPsKeys) store_key_ext(sbase + kPsOffKeyExt, tid);
    fence_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    if (warp == kPsTmaWarp) {
        if (lane == 0) {
            int t = 0, m = 0;  // row tiles and items so far
            bool ok = true;
            for (int64_t r = 0; ok && snake(r) < p.items; ++r) {
                const Item it(p, snake(r), kv);
                const RowTiles rt(p, it.k0, (it.n_heads + per_tile - 1) / per_tile);
                if (rt.n == 0) continue;
                if (m >= 1 && !mbar_wait(BAR(kPsBarKEmpty), (uint32_t)(m - 1) & 1u, abort_flag, p.status)) break;
                mbar_expect_tx(BAR(kPsBarK), 2 * kPsTile);
                for (int x = 0; x < 4; ++x)
                    tma_load_3d(sbase + x * kPsBox, &tk, 64 * (x & 1), it.k0 + kPsKeys * (x >> 1), it.bh, BAR(kPsBarK));
                ++m;
                int ht = 0, q = 0;  // head group and row tile
                for (int i = 0; i < rt.n; ++i, ++t) {
                    const int s = t % kPsStages;
                    if (t >= kPsStages && !mbar_wait(BAR(kPsBarQEmpty + s), (uint32_t)(t / kPsStages - 1) & 1u, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    mbar_expect_tx(BAR(kPsBarQ + s), kPsTile);
                    load_row_tile(&tq, srow + s * kPsTile, p, it.bh, it.g_first, it.n_heads, ht, rt.lo + q * p.box, kPsCols,
                                  BAR(kPsBarQ + s));
                    if (++q == rt.n_rows_t) {
                        q = 0;
                        ++ht;
                    }
                }
            }
            // every copy issued has landed before the CTA ends
            if (m > 0) mbar_wait(BAR(kPsBarK), (uint32_t)(m - 1) & 1u, abort_flag, p.status, false);
            for (int i = max(0, t - kPsStages); i < t; ++i)
                mbar_wait(BAR(kPsBarQ + i % kPsStages), (uint32_t)(i / kPsStages) & 1u, abort_flag, p.status, false);
        }
        __syncwarp();
    } else if (warp == kPsMmaWarp) {
        constexpr uint32_t idS = instr_desc(kPsKeys, kPsCols, 0);
        const uint32_t acc0 = __shfl_sync(0xffffffffu, tmem, 0);
        int t = 0, m = 0;
        bool ok = true;
        auto wait = [&](int bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(BAR(bar), parity & 1u, abort_flag, p.status));
        };
        for (int64_t r = 0; ok && snake(r) < p.items; ++r) {
            const Item it(p, snake(r), kv);
            const RowTiles rt(p, it.k0, (it.n_heads + per_tile - 1) / per_tile);
            if (rt.n == 0) continue;
            ok = wait(kPsBarK, (uint32_t)m);
            for (int i = 0; ok && i < rt.n; ++i, ++t) {
                const int s = t % kPsStages, b = t & 1;
                ok = wait(kPsBarQ + s, (uint32_t)(t / kPsStages)) && wait(kPsBarExt + b, (uint32_t)(t >> 1)) &&
                     (t < 2 || wait(kPsBarFree + b, (uint32_t)((t >> 1) - 1)));
                if (!ok) break;
                tc_fence_after();
                const uint32_t qa = srow + s * kPsTile, acc = acc0 + (uint32_t)(2 * kPsCols * b);
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) {
                    const uint32_t off = (uint32_t)(k >> 2) * kPsBox + (uint32_t)(k & 3) * 32;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        mma_ss_warp(acc + (uint32_t)(kPsCols * j), smem_desc(sbase + j * kPsTile + off, 16, 1024),
                                    smem_desc(qa + off, 16, 1024), idS, k > 0);
                }
                // (the ninth step last: the sum is large only then, and the
                // tensor cores' roundings go by its size)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    mma_ss_warp(acc + (uint32_t)(kPsCols * j), smem_desc(sbase + kPsOffKeyExt, 16, 1024),
                                smem_desc(sbase + kPsOffRowExt + b * kPsBox, 16, 1024), idS, 1);
                mma_commit_warp(BAR(kPsBarS + b));
                mma_commit_warp(BAR(kPsBarQEmpty + s));
            }
            if (ok) mma_commit_warp(BAR(kPsBarKEmpty));
            ++m;
        }
        // every MMA issued has completed before the CTA ends
        mma_commit_warp(BAR(kPsBarDrain));
        mbar_wait(BAR(kPsBarDrain), 0, abort_flag, p.status, false);
        __syncwarp();
    } else {
        const int w = warp >> 2, b = w >> 1, j = w & 1, r128 = tid & 127;
        const uint32_t tS = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)(kPsCols * w);
        const uint64_t c2 = pack2(p.scale_log2, p.scale_log2);
        const int box_mask = p.box - 1, box_shift = 31 - __clz(p.box);
        int t = 0, m = 0;  // row tiles and items so far
        bool dead = false;  // a wait gave up: the warp only keeps its barriers
        for (int64_t r = 0; snake(r) < p.items; ++r, ++m) {
            const Item it(p, snake(r), kv);
            const RowTiles rt(p, it.k0, (it.n_heads + per_tile - 1) / per_tile);
            const int kb = it.k0 + kPsKeys * j, key = kb + r128;  // key of the thread's lane
            const float* lse = p.lse + (size_t)it.bh * p.G * (size_t)p.T;
            // log-sum-exp of this thread's row of the item's tile i
            auto row_of = [&](int i) -> float {
                const int ht = i / rt.n_rows_t, g = ht * per_tile + (r128 >> box_shift);
                return row_lse(p, lse + (size_t)(it.g_first + min(g, it.n_heads - 1)) * p.T,
                               rt.lo + (i - ht * rt.n_rows_t) * p.box + (r128 & box_mask), g < it.n_heads);
            };
            // warpgroup 2 b writes the box of parity b for a tile as soon as
            // the columns of the last tile that used it are there
            auto write_ext = [&](float x) {
                store_ext(sbase + kPsOffRowExt + b * kPsBox, r128, row_ext(p, x));
                fence_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(kPsBarExt + b));
            };
            const int i0 = (t & 1) == b ? 0 : 1;  // the item's first tile of this parity
            if (j == 0 && !dead && i0 < rt.n) write_ext(row_of(i0));
            float sum = 0.0f;
            for (int i = i0; i < rt.n; i += 2) {
                const int u = (t + i) >> 1;  // the accumulator's tiles so far
                const float next = j == 0 && i + 2 < rt.n ? row_of(i + 2) : 0.0f;
                if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(BAR(kPsBarS + b), (uint32_t)u & 1u, abort_flag, p.status));
                if (dead) break;
                tc_fence_after();
                if (j == 0 && i + 2 < rt.n) write_ext(next);
                const int ht = i / rt.n_rows_t, r0 = rt.lo + (i - ht * rt.n_rows_t) * p.box;
                const bool edge = r0 < kb + kPsKeys - 1 || r0 + box_mask >= kb + p.window;
                const int c_lo = key - r0, c_hi = key < p.sinks ? INT32_MAX : key + p.window - r0;
                sum += edge ? sum_columns<kPsCols, true>(tS, c2, 0, box_mask, c_lo, c_hi, BAR(kPsBarFree + b))
                            : sum_columns<kPsCols, false>(tS, c2, 0, box_mask, c_lo, c_hi, BAR(kPsBarFree + b));
            }
            t += rt.n;
            // the odd row tiles' sums join the even ones' (the buffer is
            // written again two items on, past another such barrier)
            if (b == 1) s_half[j][m & 1][r128] = sum;
            bar_sync(1 + j, 256);
            if (b == 0 && key < p.T) {
                float* dst = p.parts > 1 ? p.out + ((size_t)it.bh * p.parts + it.part) * (size_t)p.T : p.out + (size_t)it.bh * (size_t)p.stride;
                dst[key] = sum + s_half[j][m & 1][r128];
            }
        }
    }
#undef BAR
    tc_fence_before();
    __syncthreads();
    if (warp == kPsMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(4 * kPsCols));
    }
}

// scores[b][h][t] = the parts' sums, in order.
__global__ void __launch_bounds__(256) prefill_score_join_kernel(const float* part, float* out, int64_t stride, int T, int parts) {
    const int t = blockIdx.x * 256 + threadIdx.x;
    const size_t unit = blockIdx.y;
    if (t >= T) return;
    float s = 0.0f;
    for (int i = 0; i < parts; ++i) s += part[(unit * parts + i) * (size_t)T + t];
    out[unit * (size_t)stride + t] = s;
}

// ---- the rows stay: CTA c of a KV head's gridDim.x takes the key tiles c, c +
// gridDim.x, ...; N = 256 columns, or 128 when those hold all the rows.
constexpr int kPrStages = 3;  // key tiles in shared memory
template <int N>
struct PrLayout {  // the rows, the key tiles, the ninth step's boxes (rows, keys)
    static constexpr uint32_t kRows = (uint32_t)N * kD * 2, kRowBox = kRows / 2;
    static constexpr uint32_t kOffKey = kRows, kOffRowExt = kOffKey + kPrStages * kPsTile, kOffKeyExt = kOffRowExt + kRowBox;
    static constexpr uint32_t kBytes = kOffKeyExt + kPsBox + 1024;
};
enum { kPrBarQ = 0, kPrBarFull = 1, kPrBarEmpty = 4, kPrBarS = 7, kPrBarFree = 9, kPrBarDrain = 11, kPrNumBars = 12 };

// The descriptors both kernels build, checked field by field for a 1
// KB-aligned base anywhere in the 227 KB a CTA can address.
bool ps_descriptors_valid() {
    if (!instr_desc_ok(instr_desc(kPsKeys, 128, 0), 0) || !instr_desc_ok(instr_desc(kPsKeys, 256, 0), 0)) return false;
    constexpr uint32_t most = kPsSmem > PrLayout<256>::kBytes ? kPsSmem : PrLayout<256>::kBytes;
    static_assert(most <= 227u * 1024u - 4096u, "beside the static shared memory");
    for (uint32_t base = 0; base + most <= 227u * 1024u + 1024; base += 1024)
        for (uint32_t at = 0; at < most - 1024; at += kPsBox)  // every box of either kernel starts at a multiple of it
            for (uint32_t off = 0; off < 128; off += 32)
                if (!smem_desc_ok(base + at + off, 16, 1024)) return false;
    return true;
}

template <int N>
__global__ void __launch_bounds__(kPsThreads, 1)
    prefill_score_rows_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk, PsParams p) {
    using PL = PrLayout<N>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_bar[kPrNumBars];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ float s_half[2][2][kPsKeys];  // [accumulator][use parity]: the sums of its upper columns
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u, skey = sbase + PL::kOffKey;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bh = (int)blockIdx.y;
    const int n_kt = (p.T + kPsKeys - 1) / kPsKeys;
    const uint32_t bar0 = smem_u32(&s_bar[0]);
    volatile int* abort_flag = &s_abort;
#define BAR(i) (bar0 + 8u * (uint32_t)(i))
    // whether a row sees a key of tile kt
    auto live = [&](int kt) -> bool {
        const int k0 = kt * kPsKeys;
        return p.row0 < p.T && (p.sinks > k0 || (int64_t)k0 + kPsKeys - 1 + p.window > p.row0);
    };

    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < kPrNumBars; ++i) mbar_init(BAR(i), (i == kPrBarFree || i == kPrBarFree + 1) ? 8 : 1);  // (8 warps)
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kPsMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(2 * N));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    const float* lse = p.lse + (size_t)bh * p.G * (size_t)p.T;
    for (int i = tid; i < N; i += kPsThreads) {
        const int g = i / p.box;
        store_ext(sbase + PL::kOffRowExt, i, row_ext(p, row_lse(p, lse + (size_t)min(g, p.G - 1) * p.T, p.row0 + i % p.box, g < p.G)));
    }
    if (tid < kPsKeys) store_key_ext(sbase + PL::kOffKeyExt, tid);
    fence_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    if (warp == kPsTmaWarp) {
        if (lane == 0) {
            mbar_expect_tx(BAR(kPrBarQ), PL::kRows);
            load_row_tile(&tq, sbase, p, bh, 0, p.G, 0, p.row0, N, BAR(kPrBarQ));
            int n = 0;  // live tiles so far
            for (int kt = blockIdx.x; kt < n_kt; kt += gridDim.x) {
                if (!live(kt)) continue;
                const int s = n % kPrStages;
                if (n >= kPrStages && !mbar_wait(BAR(kPrBarEmpty + s), (uint32_t)(n / kPrStages - 1) & 1u, abort_flag, p.status)) break;
                mbar_expect_tx(BAR(kPrBarFull + s), kPsTile);
                for (int x = 0; x < 2; ++x)
                    tma_load_3d(skey + s * kPsTile + x * kPsBox, &tk, 64 * x, kt * kPsKeys, bh, BAR(kPrBarFull + s));
                ++n;
            }
            // every copy issued has landed before the CTA ends
            mbar_wait(BAR(kPrBarQ), 0, abort_flag, p.status, false);
            for (int i = max(0, n - kPrStages); i < n; ++i)
                mbar_wait(BAR(kPrBarFull + i % kPrStages), (uint32_t)(i / kPrStages) & 1u, abort_flag, p.status, false);
        }
        __syncwarp();
    } else if (warp == kPsMmaWarp) {
        constexpr uint32_t idS = instr_desc(kPsKeys, N, 0);
        const uint32_t acc0 = __shfl_sync(0xffffffffu, tmem, 0);
        auto wait = [&](int bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(BAR(bar), parity & 1u, abort_flag, p.status));
        };
        bool ok = wait(kPrBarQ, 0);
        int n = 0;
        for (int kt = blockIdx.x; ok && kt < n_kt; kt += gridDim.x) {
            if (!live(kt)) continue;
            const int s = n % kPrStages, a = n & 1;
            ok = wait(kPrBarFull + s, (uint32_t)(n / kPrStages)) && (n < 2 || wait(kPrBarFree + a, (uint32_t)((n >> 1) - 1)));
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc = acc0 + (uint32_t)(N * a), ka = skey + s * kPsTile;
#pragma unroll
            for (int k = 0; k < kD / 16; ++k) {
                const uint32_t x = (uint32_t)(k >> 2), off = (uint32_t)(k & 3) * 32;
                mma_ss_warp(acc, smem_desc(ka + x * kPsBox + off, 16, 1024), smem_desc(sbase + x * PL::kRowBox + off, 16, 1024), idS, k > 0);
            }
            mma_ss_warp(acc, smem_desc(sbase + PL::kOffKeyExt, 16, 1024), smem_desc(sbase + PL::kOffRowExt, 16, 1024), idS, 1);
            mma_commit_warp(BAR(kPrBarS + a));
            mma_commit_warp(BAR(kPrBarEmpty + s));
            ++n;
        }
        mma_commit_warp(BAR(kPrBarDrain));
        mbar_wait(BAR(kPrBarDrain), 0, abort_flag, p.status, false);
        __syncwarp();
    } else {
        constexpr int kHalf = N / 2;
        const int w = warp >> 2, a = w >> 1, col0 = kHalf * (w & 1), r = tid & 127;
        const uint32_t tS = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)(N * a + col0);
        const uint64_t c2 = pack2(p.scale_log2, p.scale_log2);
        const int box_mask = p.box - 1;
        float* out = p.out + (size_t)bh * (size_t)p.stride;
        int n = 0;
        bool dead = false;  // a wait gave up: the warp only keeps its barriers
        for (int kt = blockIdx.x; kt < n_kt; kt += gridDim.x) {
            const int k0 = kt * kPsKeys, key = k0 + r;
            if (!live(kt)) {
                if (w == 0 && key < p.T) out[key] = 0.0f;
                continue;
            }
            if ((n++ & 1) != a) continue;
            const int u = (n - 1) >> 1;  // the accumulator's tiles so far
            if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(BAR(kPrBarS + a), (uint32_t)u & 1u, abort_flag, p.status));
            float sum = 0.0f;
            if (!dead) {
                tc_fence_after();
                const bool edge = p.row0 < k0 + kPsKeys - 1 || p.row0 + box_mask >= k0 + p.window;
                const int c_lo = key - p.row0, c_hi = key < p.sinks ? INT32_MAX : key + p.window - p.row0;
                sum = edge ? sum_columns<kHalf, true>(tS, c2, col0, box_mask, c_lo, c_hi, BAR(kPrBarFree + a))
                           : sum_columns<kHalf, false>(tS, c2, col0, box_mask, c_lo, c_hi, BAR(kPrBarFree + a));
            }
            // the upper columns' sums join the lower ones' (the buffer is
            // written again two tiles on, past another such barrier)
            if (w & 1) s_half[a][u & 1][r] = sum;
            bar_sync(1 + a, 256);
            if (!(w & 1) && key < p.T) out[key] = sum + s_half[a][u & 1][r];
        }
    }
#undef BAR
    tc_fence_before();
    __syncthreads();
    if (warp == kPsMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * N));
    }
}

struct PsPlan {
    int box, parts, heads;
    bool resident;   // the rows stay in shared memory (prefill_score_rows_kernel)
    int cols, ctas;  // resident: columns (128 or 256), CTAs per KV head
};

PsPlan ps_plan(const bgtq_plan& pl, int batch, int t, int row0) {
    PsPlan s;
    s.box = 2 * kPsCols;
    while (s.box > 16 && s.box / 2 >= t - row0) s.box /= 2;
    const int sms = pl.num_sms > 0 ? pl.num_sms : 152;  // (a host-only plan: GB300's)
    const int64_t n_kt = (t + kPsKeys - 1) / kPsKeys, kv = std::max<int64_t>(1, (int64_t)batch * pl.H);
    // all the rows in one tile: they stay, the key tiles stream.  CTAs per KV
    // head: the fewest rounds of key tiles over the waves of CTAs (a
    // CTA's start costs about two key tiles)
    s.resident = t - row0 <= s.box && pl.G * s.box <= 256;
    s.cols = pl.G * s.box <= 128 ? 128 : 256;
    s.ctas = 1;
    if (s.resident) {
        int64_t best = INT64_MAX;
        for (int64_t c = 1; c <= std::min<int64_t>(n_kt, sms); ++c) {
            const int64_t cost = (kv * c + sms - 1) / sms * ((n_kt + c - 1) / c + 2);
            if (cost < best) {
                best = cost;
                s.ctas = (int)c;
            }
        }
        s.parts = 1;
        s.heads = pl.G;
        return s;
    }
    // the query heads stay together (a key tile is loaded once) when the pairs
    // of key tiles alone are several items for every CTA or an item has few
    // row tiles; else they are shared out
    s.box = std::min(s.box, kPsCols);
    const int per_tile = kPsCols / s.box;
    const int64_t units = kv * ((n_kt + 1) / 2);
    s.heads = pl.G;
    const int64_t want = 4 * (int64_t)sms;
    const int64_t row_tiles = (t - row0 + s.box - 1) / s.box;
    while (s.heads > per_tile && units * ((pl.G + s.heads - 1) / s.heads) < want &&
           (s.heads + per_tile - 1) / per_tile * row_tiles > 8)
        s.heads = std::max(per_tile, (s.heads + 1) / 2);
    s.heads = std::min(s.heads, pl.G);
    s.parts = (pl.G + s.heads - 1) / s.heads;
    return s;
}

}  // namespace

size_t prefill_score_workspace_bytes(const bgtq_plan& pl, int batch, int t, int row0) {
    const PsPlan s = ps_plan(pl, batch, t, row0);
    return s.parts > 1 ? (size_t)batch * pl.H * s.parts * (size_t)t * sizeof(float) : 0;
}

cudaError_t launch_prefill_score(const bgtq_plan& pl, cudaStream_t s, const void* q, const void* k, const float* lse,
                                 int batch, int t, int row0, int sinks, int window, float scale, float* scores,
                                 int64_t stride, void* ws, int32_t* status) {
    static std::mutex mu;
    static bool done[64] = {false};
    static const bool desc_ok = ps_descriptors_valid();
    if (!desc_ok) return cudaErrorInvalidValue;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!done[dev]) {
            cudaError_t e =
                cudaFuncSetAttribute(prefill_score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPsSmem);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(prefill_score_rows_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)PrLayout<128>::kBytes);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(prefill_score_rows_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)PrLayout<256>::kBytes);
            if (e != cudaSuccess) return e;
            done[dev] = true;
        }
    }
    const PsPlan sp = ps_plan(pl, batch, t, row0);
    alignas(64) CUtensorMap tq, tk;
    if (!heads_map(&tq, q, (uint64_t)batch * pl.H * pl.G, t, (uint32_t)std::min(sp.box, 128)) ||
        !heads_map(&tk, k, (uint64_t)batch * pl.H, t, kPsKeys))
        return cudaErrorInvalidValue;
    PsParams p;
    p.lse = lse;
    p.out = sp.parts > 1 ? static_cast<float*>(ws) : scores;
    p.stride = stride;
    p.T = t;
    p.H = pl.H;
    p.G = pl.G;
    p.row0 = row0;
    p.sinks = sinks;
    p.window = window;
    p.box = sp.box;
    p.parts = sp.parts;
    p.heads = sp.heads;
    p.scale_log2 = scale * 1.4426950408889634f;
    const double unit = 1.0 / (double)scale;
    p.unit_hi = (float)unit;
    p.unit_lo = (float)(unit - (double)p.unit_hi);
    p.status = status;
    if (sp.resident) {
        const dim3 rg((unsigned)sp.ctas, (unsigned)((int64_t)batch * pl.H), 1);
        if (sp.cols == 256)
            prefill_score_rows_kernel<256><<<rg, kPsThreads, PrLayout<256>::kBytes, s>>>(tq, tk, p);
        else
            prefill_score_rows_kernel<128><<<rg, kPsThreads, PrLayout<128>::kBytes, s>>>(tq, tk, p);
        return cudaGetLastError();
    }
    const int kv = batch * pl.H;
    p.items = (int64_t)kv * sp.parts * ((t + 2 * kPsKeys - 1) / (2 * kPsKeys));
    const unsigned ctas = (unsigned)std::min<int64_t>(p.items, std::max(1, pl.num_sms));
    prefill_score_kernel<<<ctas, kPsThreads, kPsSmem, s>>>(tq, tk, p, kv);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || sp.parts == 1) return e;
    const dim3 jg((unsigned)((t + 255) / 256), (unsigned)((int64_t)batch * pl.H), 1);
    prefill_score_join_kernel<<<jg, 256, 0, s>>>(static_cast<const float*>(ws), scores, stride, t, sp.parts);
    return cudaGetLastError();
}

}  // namespace bgtq
