// Accumulated attention weights of a prompt's rows: for every key j of a KV
// head, the sum over the head's query heads and the rows i >= row0 of
//   exp(scale q_i . k_j - lse_i),   j <= i and (j < sinks or j > i - window),
// from the rows' log-sum-exp (bgtq_prefill_window_attn writes it).  These are
// the scores that rank the positions of a cache before it is cut to a budget.
//
// One pass over the (row, key) pairs, no softmax statistics to find: S^T =
// K_tile Q_tile^T on the tensor cores (tcgen05, keys in the 128 tensor-memory
// lanes, rows in the columns), so that a thread owns a key and its sum stays
// in a register over all rows: no reduction between threads, no atomics.
// Per pair the tensor cores do 256 flop and the SM one exponential; at 16
// exponentials a clock a 128 x 128 tile takes 1024 clocks against about 512 of
// MMAs, so the exponentials bound it.
//
// CTA: one key tile of one KV head and a share of its query heads; 10 warps:
//   warps 0-3, 4-7  warpgroups that take the row tiles in turn: thread = key =
//                   tensor-memory lane, 128 columns of the tile's S^T
//   warp 8          issues the MMAs (one thread), owns the tensor memory (256
//                   columns: an accumulator per warpgroup)
//   warp 9          issues the TMA copies (one thread): the key tile once, row
//                   tiles through two stages
// 97 KB of shared memory and 256 columns: two CTAs per SM, so that one's
// set-up and tail run under the other's tiles.  Where few rows count (at most
// 64), a tile of 128 columns is filled with the rows of several query heads.
// Rows that do not count get a weight exponent of -inf with their lse.  With
// few key tiles the query heads are shared out over several CTAs, whose sums
// a second kernel adds in order.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "tc_common.cuh"

namespace bgtq {
namespace {

constexpr int kPsKeys = 128, kPsCols = 128;
constexpr int kPsGroups = 2;                                 // warpgroups = tensor-memory accumulators
constexpr int kPsThreads = kPsGroups * 128 + 64;
constexpr int kPsStages = 2;
constexpr uint32_t kPsTile = 128 * kD * 2;                   // 32 KB
constexpr uint32_t kPsBox = kPsTile / 2;                     // a 64-column box of it
constexpr uint32_t kPsSmem = (1 + kPsStages) * kPsTile + 1024;
constexpr uint32_t kPsTmem = kPsGroups * kPsCols;

enum { kPsBarK = 0, kPsBarFull = 1, kPsBarEmpty = 3, kPsBarS = 5, kPsBarFree = 7, kPsBarDrain = 9, kPsNumBars = 10 };

struct PsParams {
    const float* lse;  // [B][H*G][T]
    float* out;        // [B][H][stride] or, with parts > 1, [B][H][parts][T]
    int64_t stride;
    int T, H, G, row0, sinks, window;
    int box;           // rows of a TMA box: 128, or fewer with several heads in a tile
    int parts, heads;  // CTAs per key tile, query heads of each
    float scale_log2;
    int32_t* status;
};

bool ps_descriptors_valid() {
    if (!instr_desc_ok(instr_desc(kPsKeys, kPsCols, 0), 0)) return false;
    for (uint32_t base = 0; base + kPsSmem <= 227u * 1024u + 1024; base += 1024)
        for (int st = 0; st <= kPsStages; ++st)
            for (int k = 0; k < kD / 16; ++k)
                if (!smem_desc_ok(base + st * kPsTile + (uint32_t)(k >> 2) * kPsBox + (uint32_t)(k & 3) * 32, 16, 1024)) return false;
    return true;
}

// The row tiles of a key tile: rows lo + 128 r.., for each group of query heads.
struct RowTiles {
    int lo, n_rows_t, n;
    __device__ __forceinline__ RowTiles(const PsParams& p, int k0, int n_head_t) {
        lo = max(p.row0, k0);
        const int hi = p.sinks > k0 ? p.T : (int)min((int64_t)p.T, (int64_t)k0 + kPsKeys - 1 + p.window);
        n_rows_t = hi > lo ? (hi - lo + p.box - 1) / p.box : 0;
        n = n_rows_t * n_head_t;
    }
};

// Barrier kId of a warpgroup; true if every thread's `ok` is.
template <int kId>
__device__ __forceinline__ bool group_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.and.pred q, %1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "n"(kId), "r"((uint32_t)ok)
        : "memory");
    return r != 0;
}

__global__ void __launch_bounds__(kPsThreads, 2)
    prefill_score_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk, PsParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_bar[kPsNumBars];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ __align__(16) float s_nlse[kPsGroups][2][kPsCols];  // -lse log2 e of a tile's columns
    __shared__ float s_sum[kPsKeys];
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int part = (int)blockIdx.x % p.parts;
    const int h = (int)(blockIdx.x / p.parts) % p.H;
    const int b = (int)blockIdx.x / (p.parts * p.H);
    const int k0 = (int)blockIdx.y * kPsKeys;
    const int g_first = part * p.heads, n_heads = min(p.heads, p.G - g_first);
    const int per_tile = kPsCols / p.box;                       // query heads of a tile
    const RowTiles rt(p, k0, (n_heads + per_tile - 1) / per_tile);
    const uint32_t bar0 = smem_u32(&s_bar[0]);
    volatile int* abort_flag = &s_abort;
#define BAR(i) (bar0 + 8u * (uint32_t)(i))

    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < kPsNumBars; ++i) mbar_init(BAR(i), (i == kPsBarFree || i == kPsBarFree + 1) ? 128 : 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(kPsTmem));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    float sum = 0.0f;

    if (warp == 9) {
        if (lane == 0 && rt.n > 0) {
            int used[kPsStages] = {0, 0};  // tiles issued on each stage
            mbar_expect_tx(BAR(kPsBarK), kPsTile);
            for (int x = 0; x < 2; ++x)
                tma_load_2d(sbase + x * kPsBox, &tk, 64 * x, (b * p.H + h) * p.T + k0, BAR(kPsBarK));
            int ht = 0, r = 0;  // head group and row tile of tile t
            for (int t = 0; t < rt.n; ++t) {
                const int s = t & 1;
                if (t >= kPsStages && !mbar_wait(BAR(kPsBarEmpty + s), (uint32_t)((t >> 1) - 1) & 1u, abort_flag, p.status)) break;
                mbar_expect_tx(BAR(kPsBarFull + s), kPsTile);
                for (int u = 0; u < per_tile; ++u) {
                    // (a head group's last tile may have too few heads: the last one again, not counted)
                    const int g = g_first + min(ht * per_tile + u, n_heads - 1);
                    const int y = ((b * p.H + h) * p.G + g) * p.T + rt.lo + r * p.box;
                    for (int x = 0; x < 2; ++x)
                        tma_load_2d(sbase + (1 + s) * kPsTile + x * kPsBox + (uint32_t)(u * p.box) * 128u, &tq, 64 * x, y,
                                    BAR(kPsBarFull + s));
                }
                used[s] = (t >> 1) + 1;
                if (++r == rt.n_rows_t) {
                    r = 0;
                    ++ht;
                }
            }
            // every copy issued has landed before the CTA ends
            mbar_wait(BAR(kPsBarK), 0, abort_flag, p.status, false);
            for (int s = 0; s < kPsStages; ++s)
                if (used[s]) mbar_wait(BAR(kPsBarFull + s), (uint32_t)(used[s] - 1) & 1u, abort_flag, p.status, false);
        }
        __syncwarp();
    } else if (warp == 8) {
        if (lane == 0 && rt.n > 0) {
            constexpr uint32_t idS = instr_desc(kPsKeys, kPsCols, 0);
            bool ok = mbar_wait(BAR(kPsBarK), 0, abort_flag, p.status);
            for (int t = 0; ok && t < rt.n; ++t) {
                const int s = t & 1;  // stage and accumulator
                const uint32_t par = (uint32_t)(t >> 1) & 1u;
                ok = mbar_wait(BAR(kPsBarFull + s), par, abort_flag, p.status) &&
                     (t < kPsGroups || mbar_wait(BAR(kPsBarFree + s), par ^ 1u, abort_flag, p.status));
                if (!ok) break;
                tc_fence_after();
                const uint32_t qa = sbase + (1 + s) * kPsTile;
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) {
                    const uint32_t off = (uint32_t)(k >> 2) * kPsBox + (uint32_t)(k & 3) * 32;
                    mma_ss(tmem + (uint32_t)kPsCols * s, smem_desc(sbase + off, 16, 1024), smem_desc(qa + off, 16, 1024), idS, k > 0);
                }
                mma_commit(BAR(kPsBarS + s));
                mma_commit(BAR(kPsBarEmpty + s));
            }
            mma_commit(BAR(kPsBarDrain));
            mbar_wait(BAR(kPsBarDrain), 0, abort_flag, p.status, false);
        }
        __syncwarp();
    } else {
        const int w = warp >> 2, col = tid & 127;
        const int key = k0 + col;  // lane of the tensor memory
        const uint32_t tS = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)kPsCols * w;
        const float c = p.scale_log2;
        const float* lse = p.lse + ((size_t)b * p.H + h) * p.G * (size_t)p.T;
        const int box_mask = p.box - 1, box_shift = 31 - __clz(p.box);
        // exponent offset of this thread's column in tile t
        auto column = [&](int t) -> float {
            const int ht = t / rt.n_rows_t, r = t - ht * rt.n_rows_t;
            const int g = ht * per_tile + (col >> box_shift), row = rt.lo + r * p.box + (col & box_mask);
            if (g >= n_heads || row >= p.T) return -INFINITY;
            const float x = __ldg(lse + (size_t)(g_first + g) * p.T + row);
            return x > -INFINITY ? -x * 1.4426950408889634f : -INFINITY;  // a row that saw nothing gives nothing
        };
        float next = w < rt.n ? column(w) : 0.0f;
        for (int t = w; t < rt.n; t += kPsGroups) {
            float* buf = s_nlse[w][(t >> 1) & 1];
            buf[col] = next;
            if (t + kPsGroups < rt.n) next = column(t + kPsGroups);
            // one barrier of the warpgroup orders the offsets and makes go or
            // stop one decision of its 128 threads
            const bool ok = mbar_wait(BAR(kPsBarS + w), (uint32_t)(t >> 1) & 1u, abort_flag, p.status);
            if (!(w == 0 ? group_all<1>(ok) : group_all<2>(ok))) break;
            tc_fence_after();
            const int ht = t / rt.n_rows_t, r0 = rt.lo + (t - ht * rt.n_rows_t) * p.box;
            // columns (rows of the box) that see the key: [c_lo, c_hi)
            const int c_lo = key - r0, c_hi = key < p.sinks ? INT32_MAX : key + p.window - r0;
            const bool edge = r0 < k0 + kPsKeys - 1 || r0 + box_mask >= k0 + p.window;
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < kPsCols / 64; ++q) {
                float s[64];
                tmem_ld32(tS + 64 * q, s);
                tmem_ld32(tS + 64 * q + 32, s + 32);
                tmem_wait_ld32(s);
                tmem_wait_ld32(s + 32);
                if (q == kPsCols / 64 - 1) {  // the accumulator is read: the next tile may overwrite it
                    tc_fence_before();
                    mbar_arrive(BAR(kPsBarFree + w));
                }
                if (edge) {
#pragma unroll
                    for (int i = 0; i < 64; ++i) {
                        const int cc = (64 * q + i) & box_mask;
                        if (cc < c_lo || cc >= c_hi) s[i] = -INFINITY;
                    }
                }
                const float4* nl = reinterpret_cast<const float4*>(buf + 64 * q);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float4 n4 = nl[i];
                    acc[0] += ex2(fmaf(s[4 * i], c, n4.x));
                    acc[1] += ex2(fmaf(s[4 * i + 1], c, n4.y));
                    acc[2] += ex2(fmaf(s[4 * i + 2], c, n4.z));
                    acc[3] += ex2(fmaf(s[4 * i + 3], c, n4.w));
                }
            }
            sum += (acc[0] + acc[1]) + (acc[2] + acc[3]);
        }
        if (w == 1) s_sum[col] = sum;
    }
#undef BAR
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kPsTmem));
    }
    if (tid < kPsKeys && k0 + tid < p.T) {
        const size_t unit = (size_t)b * p.H + h;
        float* dst = p.parts > 1 ? p.out + (unit * p.parts + part) * (size_t)p.T : p.out + unit * (size_t)p.stride;
        dst[k0 + tid] = sum + s_sum[tid];
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

struct PsPlan {
    int box, parts, heads;
};

PsPlan ps_plan(const bgtq_plan& pl, int batch, int t, int row0) {
    PsPlan s;
    s.box = 128;
    while (s.box > 16 && s.box / 2 >= t - row0) s.box /= 2;
    const int per_tile = kPsCols / s.box;
    // the query heads stay together (the key tile is loaded once, no second
    // kernel) when the key tiles alone fill the GPU several times over or a
    // CTA has few row tiles; else they are shared out
    const int64_t units = (int64_t)batch * pl.H * ((t + kPsKeys - 1) / kPsKeys);
    s.heads = pl.G;
    const int64_t want = 8 * (int64_t)(pl.num_sms > 0 ? pl.num_sms : 152);  // (a host-only plan: GB300's)
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
            const cudaError_t e =
                cudaFuncSetAttribute(prefill_score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPsSmem);
            if (e != cudaSuccess) return e;
            done[dev] = true;
        }
    }
    const PsPlan sp = ps_plan(pl, batch, t, row0);
    alignas(64) CUtensorMap tq, tk;
    if (!rows_map(&tq, q, (uint64_t)batch * pl.H * pl.G * t, (uint32_t)sp.box) ||
        !rows_map(&tk, k, (uint64_t)batch * pl.H * t, kPsKeys))
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
    p.status = status;
    const dim3 grid((unsigned)((int64_t)batch * pl.H * sp.parts), (unsigned)((t + kPsKeys - 1) / kPsKeys), 1);
    prefill_score_kernel<<<grid, kPsThreads, kPsSmem, s>>>(tq, tk, p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || sp.parts == 1) return e;
    const dim3 jg((unsigned)((t + 255) / 256), (unsigned)((int64_t)batch * pl.H), 1);
    prefill_score_join_kernel<<<jg, 256, 0, s>>>(static_cast<const float*>(ws), scores, stride, t, sp.parts);
    return cudaGetLastError();
}

}  // namespace bgtq
