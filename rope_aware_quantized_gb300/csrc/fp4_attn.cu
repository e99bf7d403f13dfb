// Attention of a few query rows over the 4-bit cache in one pass over its
// bytes (up to 32 rows of a KV head: a decode step of up to 8 query heads, or
// a few drafted tokens).
//
// out = sum_j softmax_j(scale q.k_j) v_j over the positions a row sees; split
// over the positions, one running maximum and sum per warp, partials joined by
// log-sum-exp.  A warp takes pairs of groups (32 positions), brought to shared
// memory by bulk copies, kStages pairs in flight a warp.  Of each group:
//   S^T = K Q^T   (16 positions x 8 rows, K 16 dims a step): codes to fp16 by
//                 the hardware's conversion, times the block's scale, exact;
//                 the products are fp16 x fp16 in fp32
//   P^T           exp2(scaled S - m) in fp32, summed, then rounded to fp16 (fp16
//                 outputs) or split into two fp16 parts, 22 bits (fp32 outputs),
//                 transposed from accumulator to operand by movmatrix
//   O^T += V^T P^T  (16 dims x 8 rows, 16 positions a step), for each part
// One part where the output is rounded to fp16 itself: an output is then off
// by 2.6e-4 (2-norm) instead of 2.1e-4, and 32 x 8 heads of up to 16384 take
// 69 us instead of 76.
// A lane's operands are contiguous in a group (that is its layout), so a
// group is read with eight conflict-free loads a lane.  mma.sync, not tcgen05:
// 8 to 32 rows a head leave a 128-row tile idle, and its operands would have
// to pass through shared memory once more, decoded (4.5 -> 16 bits a value).
// Two groups at a time: their chains of products and exponentials run side by
// side, and the wait, the reference's check and the loop are paid once.
// What bounds it: 32 x 8 heads of up to 16384 take 69 us, 67 % of HBM's copy rate.
// No unit is full (issue slots 60 % of the active clocks, tensor pipe 20 %): of a
// warp's time a fifth is the fixed latencies of its chain of conversions, products
// and exponentials, 16 % other warps' turns, 13 % the arithmetic pipes, 11 %
// barriers, 5 % loads.  Two heads of 131072 take 20 us, of which 5 pass before the
// first data and 7 in the joins.
// The reference m of a row's exponentials stays kLift below the largest logit
// when set and moves only when a logit passes it by kRange, so that the parts
// keep their bits well above fp16's smallest numbers.
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "fp4.cuh"
#include "tc_common.cuh"

namespace bgtq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;         // pairs of groups in flight a warp
constexpr int kRowPad = 132;       // floats of a row of partial output in shared memory (keeps the warp's stores on 32 banks)
constexpr float kLift = 8.0f, kRange = 15.0f;
constexpr float kLow = -1.0e30f;   // "no position yet"
constexpr int kPair = 2 * kGroup, kPairBytes = 2 * kGroupBytes;
constexpr int kUnitCost = 16;      // what a unit's start and end take of a CTA, in pairs of groups

struct AttnParams {
    RopeParams rope;
    RowsView q;
    Fp4Map map;
    const int32_t* seq_lens;
    int max_len;
    int batch, t, group, H;
    int clusters;        // of the launch
    int least;           // pairs that a cluster takes at least
    bool pad;            // few units: each in whole ranges (see Share)
    void* out;
    int out_dtype;
    float scale_log2;
    uint32_t* counters;  // [cluster][rank]: arrivals at the unit that is split and begins in that cluster
    float2* part_ml;     // [cluster][2][R]: (m, l)
    float* part_o;       // [cluster][2][R][128]
    int32_t* status;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

// A warp's running state: rows 8 nq + 2 c + e (c = lane mod 4, e = 0, 1),
// dims 16 j + lane / 4 (+ 8).
template <int NQ>
struct State {
    float o[8][NQ][4];
    float m[NQ][2], l[NQ][2];
};

// The query's B operand: in registers, or (more row tiles, whose accumulators
// need them) read again from shared memory, conflict-free by the rows' padding.
constexpr int kQPad = 16;
template <int NQ>
struct Query {
    const __half* at;
    __device__ __forceinline__ void load(const __half (*rows)[kD + kQPad], int lane) { at = &rows[lane >> 2][4 * (lane & 3)]; }
    __device__ __forceinline__ uint2 get(int j, int i) const { return *reinterpret_cast<const uint2*>(at + 8 * i * (kD + kQPad) + 16 * j); }
};
template <>
struct Query<1> {
    uint2 w[8];
    __device__ __forceinline__ void load(const __half (*rows)[kD + kQPad], int lane) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = *reinterpret_cast<const uint2*>(&rows[lane >> 2][16 * j + 4 * (lane & 3)]);
    }
    __device__ __forceinline__ uint2 get(int j, int) const { return w[j]; }
};

// A pair of groups (`first`: of the warp's in this segment): img in shared
// memory, base its first position, lim the last position each of the lane's
// rows sees; kEdge: some position is not seen by every row (from n on: its
// bytes do not count).
template <int NQ, bool kTwo, bool kEdge>
__device__ __forceinline__ void attend(State<NQ>& st, bool first, const Query<NQ>& q, const uint8_t* img, int base, int n,
                                       const int (&lim)[NQ][2], float c, int lane) {
    const int g = lane >> 2, cl = lane & 3;
    float s[2][NQ][4];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < NQ; ++i) s[x][i][0] = s[x][i][1] = s[x][i][2] = s[x][i][3] = 0.0f;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const uint8_t* at = img + x * kGroupBytes;
        const uint4 ka = *reinterpret_cast<const uint4*>(at + 64 * g + 16 * cl);
        const uint4 kb = *reinterpret_cast<const uint4*>(at + 64 * (g + 8) + 16 * cl);
        const uint2 sa = *reinterpret_cast<const uint2*>(at + kGroupKs + 8 * g);
        const uint2 sb = *reinterpret_cast<const uint2*>(at + kGroupKs + 8 * (g + 8));
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            const uint32_t ta = jj < 2 ? sa.x : sa.y, tb = jj < 2 ? sb.x : sb.y;
            const __half2 ha = (jj & 1) ? fp4_scales<2>(ta) : fp4_scales<0>(ta), hb = (jj & 1) ? fp4_scales<2>(tb) : fp4_scales<0>(tb);
            __half2 xa[4], xb[4];
            fp4_numbers(wa[jj], xa);
            fp4_numbers(wb[jj], xb);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const __half2 ma = k ? __high2half2(ha) : __low2half2(ha), mb = k ? __high2half2(hb) : __low2half2(hb);
                const uint32_t a0 = h2u(__hmul2(xa[2 * k], ma)), a1 = h2u(__hmul2(xb[2 * k], mb));
                const uint32_t a2 = h2u(__hmul2(xa[2 * k + 1], ma)), a3 = h2u(__hmul2(xb[2 * k + 1], mb));
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    const uint2 w = q.get(2 * jj + k, i);
                    mma16816(s[x][i], a0, a1, a2, a3, w.x, w.y);
                }
            }
        }
    }
    // logits above the row's reference: positions g (0, 1) and g + 8 (2, 3), rows 2 cl (0, 2) and 2 cl + 1 (1, 3)
    float top = -INFINITY;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[x][i][e] = fmaf(s[x][i][e], c, -st.m[i][e & 1]);
                if (kEdge && base + kGroup * x + g + 8 * (e >> 1) > lim[i][e & 1]) s[x][i][e] = -INFINITY;
                top = fmaxf(top, s[x][i][e]);
            }
    if (first || __any_sync(0xffffffffu, top > kRange)) {
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mt = fmaxf(fmaxf(s[0][i][e], s[0][i][e + 2]), fmaxf(s[1][i][e], s[1][i][e + 2]));
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
                // (the first pair sets the reference: a row that sees nothing of the warp's
                // lowest positions sees none of its others)
                if (mt > kRange || (first && mt != -INFINITY)) {
                    const float up = mt - kLift;
                    const float f = first ? 1.0f : ex2(-up);
                    st.m[i][e] += up;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        s[x][i][e] -= up;
                        s[x][i][e + 2] -= up;
                    }
                    st.l[i][e] *= f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        st.o[j][i][e] *= f;
                        st.o[j][i][e + 2] *= f;
                    }
                }
            }
    }
    uint32_t hi[2][NQ][2], lo[2][NQ][2];  // lo: with kTwo
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const float p0 = ex2(s[x][i][2 * y]), p1 = ex2(s[x][i][2 * y + 1]);
                st.l[i][0] += p0;
                st.l[i][1] += p1;
                const __half2 h = __floats2half2_rn(p0, p1);
                hi[x][i][y] = transpose8(h2u(h));
                if constexpr (kTwo) {
                    const float2 b = __half22float2(h);
                    lo[x][i][y] = transpose8(h2u(__floats2half2_rn(p0 - b.x, p1 - b.y)));
                }
            }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const uint8_t* at = img + x * kGroupBytes;
        uint32_t dead = 0xffffffffu;  // scale bytes of positions past the sequence: their bits do not count
        if (kEdge) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (base + kGroup * x + 2 * cl + (e & 1) + 8 * (e >> 1) >= n) dead &= ~(0xffu << (8 * e));
        }
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
            const uint4 v = *reinterpret_cast<const uint4*>(at + kGroupV + 512 * jj + 16 * lane);
            const uint4 t = *reinterpret_cast<const uint4*>(at + kGroupVs + 32 * cl + 16 * jj);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w}, sc[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t u = kEdge ? sc[k] & dead : sc[k];
                const __half2 f0 = fp4_scales<0>(u), f1 = fp4_scales<2>(u);
                __half2 y[4];
                fp4_numbers(w[k], y);
                const uint32_t a0 = h2u(__hmul2(y[0], f0)), a1 = h2u(__hmul2(y[1], f0));
                const uint32_t a2 = h2u(__hmul2(y[2], f1)), a3 = h2u(__hmul2(y[3], f1));
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    mma16816(st.o[4 * jj + k][i], a0, a1, a2, a3, hi[x][i][0], hi[x][i][1]);
                    if constexpr (kTwo) mma16816(st.o[4 * jj + k][i], a0, a1, a2, a3, lo[x][i][0], lo[x][i][1]);
                }
            }
        }
    }
}

// The copies' ring and, once a segment's copies are used up, the partials: the
// warps' (kWarps x R padded rows), then those joined once (R rows).
constexpr int kRingBytes = kWarps * kStages * kPairBytes;
template <int NQ>
constexpr int partial_bytes = 8 * NQ * (kWarps * kRowPad + kD) * 4;
template <int NQ>
constexpr int smem_bytes = kRingBytes > partial_bytes<NQ> ? kRingBytes : partial_bytes<NQ>;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster_v2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}

// The work is a list of pairs of groups, unit (sequence, KV head) after unit, cut into
// equal ranges, one for each cluster of CTAs.  With few units a range is
// ceil(pairs / (clusters - units)) pairs and every unit is padded to whole
// ranges, so that a cluster has one unit and starts and ends once; with many,
// a unit is followed by kUnitCost empty places (what its start and end take of
// a CTA), and a range may hold several units and parts of two more.
// A unit in one cluster is finished there; one in several leaves a partial in
// each (the first or a later unit of the range), which the last cluster to
// arrive joins.  All of it follows from seq_lens, which every CTA sums up for
// itself.
constexpr int kTwoCtas = 1;  // row tiles up to which two CTAs share a SM (128 registers a thread)
struct Share {
    int per;    // places of a cluster
    int total;  // places of all units
    bool pad;
    __device__ __forceinline__ int places(int pairs) const {
        return pad ? (pairs + per - 1) / per * per : pairs + kUnitCost;
    }
};

template <int NQ, bool kTwo>
__global__ void __launch_bounds__(kThreads, NQ <= kTwoCtas ? 2 : 1) fp4_attn_kernel(const __grid_constant__ AttnParams p) {
    constexpr int R = 8 * NQ;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) __half s_q[R][kD + kQPad];
    __shared__ float2 s_part_ml[R], s_ml[kWarps][R];
    __shared__ int s_lim[R];
    __shared__ __align__(8) uint64_t s_bar[kWarps * kStages];
    __shared__ int s_abort, s_last;
    __shared__ int s_scan[kWarps], s_at[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cs = (int)cluster_size(), rank = (int)cluster_rank();
    const int k = (int)blockIdx.x / cs;
    const int rows = p.t * p.group, units = p.batch * p.H;  // (pad: units < clusters)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid < kWarps * kStages) mbar_init(smem_u32(&s_bar[tid]), 1);
    if (tid == 0) s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    auto seq_len = [&](int b) -> int {
        const int n = p.seq_lens[b];
        return min(max(n, 0), p.max_len);
    };
    // (a sequence without positions: one pair, so that its zeros are written)
    auto pairs_of = [](int n) -> int { return max(1, (n + kPair - 1) / kPair); };
    // ---- the cluster's range: where it begins
    Share sh;
    sh.pad = p.pad;
    int b = 0, start = 0, n = 0;  // start: places before sequence b
    {
        const int each = (p.batch + kThreads - 1) / kThreads;
        const int b0 = min(tid * each, p.batch), b1 = min(b0 + each, p.batch);
        // sum over all sequences, and before this thread's (whole block)
        auto scan = [&](int mine, int& before) -> int {
            int run = mine;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, run, x);
                if (lane >= x) run += o;
            }
            if (lane == 31) s_scan[warp] = run;
            __syncthreads();
            int all = 0;
            before = run - mine;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                if (x < warp) before += s_scan[x];
                all += s_scan[x];
            }
            return all;
        };
        int sum = 0, before = 0;
        if (p.batch == 1) {
            n = seq_len(0);
            sh.total = pairs_of(n) * p.H;
        } else {
            for (int x = b0; x < b1; ++x) sum += pairs_of(seq_len(x)) * p.H;
            sh.total = scan(sum, before);
        }
        if (sh.pad) {
            sh.per = max(p.least, (sh.total + p.clusters - units - 1) / (p.clusters - units));
            if (p.batch == 1) {
                sh.total = sh.places(pairs_of(n)) * p.H;
            } else {
                sum = 0;
                for (int x = b0; x < b1; ++x) sum += sh.places(pairs_of(seq_len(x))) * p.H;
                __syncthreads();
                sh.total = scan(sum, before);
            }
        } else {
            before += min(b0, p.batch) * p.H * kUnitCost;
            sum += (b1 - b0) * p.H * kUnitCost;
            sh.total += units * kUnitCost;
            sh.per = max(p.least, (sh.total + p.clusters - 1) / p.clusters);
        }
        const int lo = k * sh.per;
        if (p.batch > 1) {
            if (lo >= before && lo < before + sum) {
                int at = before, x = b0;
                for (;; ++x) {
                    const int g = sh.places(pairs_of(seq_len(x))) * p.H;
                    if (lo < at + g) break;
                    at += g;
                }
                s_at[0] = x;
                s_at[1] = at;
            }
            __syncthreads();
        }
        if (lo >= sh.total) return;  // (the whole cluster)
        if (p.batch > 1) {
            b = s_at[0];
            start = s_at[1];
            n = seq_len(b);
        }
    }
    const int lo = k * sh.per, hi = min(sh.total, lo + sh.per);
    int h = (lo - start) / sh.places(pairs_of(n));
    start += h * sh.places(pairs_of(n));
    __syncthreads();  // barriers initialised

    uint8_t* ring = smem + warp * (kStages * kPairBytes);
    float* so = reinterpret_cast<float*>(smem);
    float(*s_part)[kD] = reinterpret_cast<float(*)[kD]>(smem + kWarps * R * kRowPad * 4);
    const uint32_t ring_a = smem_u32(ring), bar_a = smem_u32(&s_bar[warp * kStages]);
    volatile int* abort_flag = &s_abort;
    const int g = lane >> 2, cl = lane & 3;
    int stage = 0;
    uint32_t parity = 0;
    const int step = cs * kWarps;  // warps of the cluster take the pairs in turn
    while (start < hi) {
        // ---- unit (b, h): its pairs [g0, g1) are the cluster's
        const int unit_pairs = pairs_of(n), unit_end = start + unit_pairs;
        const int next_start = start + sh.places(unit_pairs);
        const int g0 = max(lo - start, 0), seg_end = min(unit_end, hi) - start, g1 = min(seg_end, (n + kPair - 1) / kPair);
        if (g0 < seg_end) {
            const int gw = g0 + rank * kWarps + warp;
            // ---- the query rows (row r: token r / group, query head h group + r mod
            // group): a warp brings rows warp, warp + 8, ..; a lane 4 elements
            // and their partners, loads first
            uint2 qa[NQ], qb[NQ];
            int q_lim[NQ], q_pos[NQ][kMaxAxes];
            bool q_ok[NQ];
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const int r = warp + kWarps * i;
                qa[i] = qb[i] = make_uint2(0u, 0u);
                q_lim[i] = n - 1;
                q_ok[i] = true;
                if (r < rows) {
                    const int x = r / p.group, a = r - x * p.group;
                    q_lim[i] = n - p.t + x;
                    const __half* row = static_cast<const __half*>(p.q.p) + b * p.q.sb + (int64_t)(h * p.group + a) * p.q.sh + x * p.q.st;
                    qa[i] = *reinterpret_cast<const uint2*>(row + 4 * lane);
                    if (p.rope.cos) {
                        if (p.rope.layout == 0) qb[i] = *reinterpret_cast<const uint2*>(row + ((4 * lane) ^ 64));
                        q_ok[i] = rope_positions(p.rope, (int64_t)b * p.t + x, q_lim[i], q_pos[i]);
                    }
                }
            }
            // a pair's groups lie side by side, but for pages of one group and the last
            // group of an odd number
            auto fetch = [&](int gi, int st) {
                const bool both = 2 * gi + 1 < (n + kGroup - 1) / kGroup;
                const bool one_copy = both && (!p.map.page_table || p.map.lg > 0);
                mbar_expect_tx(bar_a + 8 * st, both ? kPairBytes : kGroupBytes);
                for (int x = 0; x < (both && !one_copy ? 2 : 1); ++x) {
                    const uint8_t* src = p.map.group(b, h, 2 * gi + x);
                    uint32_t bytes = one_copy ? kPairBytes : kGroupBytes;
                    if (!src) {
                        if (p.status) atomicOr(p.status, BGTQ_STATUS_PAGE_RANGE);
                        src = p.map.base;  // (the pool's first groups: the output is unspecified)
                    }
                    bulk_copy(ring_a + st * kPairBytes + x * kGroupBytes, src, bytes, bar_a + 8 * st);
                }
            };
            auto fetch_first = [&](int s0, int s1) {
                for (int s = s0; s < s1; ++s)
                    if (gw + s * step < g1) fetch(gw + s * step, (stage + s) % kStages);
            };
            // (one stage a warp before the query's cos and sin, the others after: those
            // small loads would queue behind all the warps' copies)
            if (lane == 0) fetch_first(0, 1);
            if (tid == 0 && rank == 0 && h == 0 && g0 == 0 && p.status && n != p.seq_lens[b]) {
                atomicOr(p.status, BGTQ_STATUS_SEQLEN_CAPACITY);
                debug_in_range(false, p.status);  // groups past the bound
            }
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const int r = warp + kWarps * i;
                uint2 w = qa[i];
                if (p.rope.cos && r < rows) {
                    if (q_lim[i] >= 0 && q_ok[i]) {
                        float2 x0 = rope_f2(qa[i].x), x1 = rope_f2(qa[i].y);
                        float c[4], s[4];
                        if (p.rope.layout == 0) {
                            // blocks 4 (lane mod 16) ..: this lane has one dim of each, lane ^ 16 the other
                            float2 y0 = rope_f2(qb[i].x), y1 = rope_f2(qb[i].y);
                            rope_load4(p.rope, q_pos[i], 4 * (lane & 15), c, s);
                            if (lane < 16) {
                                rope_pair(x0.x, y0.x, c[0], s[0]);
                                rope_pair(x0.y, y0.y, c[1], s[1]);
                                rope_pair(x1.x, y1.x, c[2], s[2]);
                                rope_pair(x1.y, y1.y, c[3], s[3]);
                            } else {
                                rope_pair(y0.x, x0.x, c[0], s[0]);
                                rope_pair(y0.y, x0.y, c[1], s[1]);
                                rope_pair(y1.x, x1.x, c[2], s[2]);
                                rope_pair(y1.y, x1.y, c[3], s[3]);
                            }
                        } else {
                            // blocks 2 lane and 2 lane + 1 of the four from 4 (lane / 2)
                            rope_load4(p.rope, q_pos[i], 4 * (lane >> 1), c, s);
                            const bool up = lane & 1;
                            rope_pair(x0.x, x0.y, up ? c[2] : c[0], up ? s[2] : s[0]);
                            rope_pair(x1.x, x1.y, up ? c[3] : c[1], up ? s[3] : s[1]);
                        }
                        w = make_uint2(rope_h2(x0.x, x0.y), rope_h2(x1.x, x1.y));
                    } else {
                        if (q_lim[i] >= 0 && lane == 0 && rank == 0 && p.status) atomicOr(p.status, BGTQ_STATUS_ROPE_RANGE);
                        w = make_uint2(0u, 0u);
                        q_lim[i] = -1;
                    }
                }
                *reinterpret_cast<uint2*>(&s_q[r][4 * lane]) = w;
                if (lane == 0) s_lim[r] = q_lim[i];
            }
            if (lane == 0) fetch_first(1, kStages);
            __syncthreads();
            Query<NQ> q;
            q.load(s_q, lane);
            int lim[NQ][2], lim_min = n - 1;
            State<NQ> st;
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j) st.o[j][i][0] = st.o[j][i][1] = st.o[j][i][2] = st.o[j][i][3] = 0.0f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    lim[i][e] = s_lim[8 * i + 2 * cl + e];
                    lim_min = min(lim_min, lim[i][e]);
                    st.m[i][e] = 0.0f;
                    st.l[i][e] = 0.0f;
                }
            }
            lim_min = __reduce_min_sync(0xffffffffu, lim_min);
            // ---- the pairs
            for (int gi = gw; gi < g1; gi += step) {
                if (!__all_sync(0xffffffffu, mbar_wait(bar_a + 8 * stage, parity, abort_flag, p.status))) {
                    // gave up: the warp's own copies land (or time out once more) before the CTA ends
                    for (int s = 0; s < kStages && gi + s * step < g1; ++s) {
                        mbar_wait(bar_a + 8 * stage, parity, abort_flag, p.status, false);
                        if (++stage == kStages) {
                            stage = 0;
                            parity ^= 1u;
                        }
                    }
                    break;
                }
                const uint8_t* img = ring + stage * kPairBytes;
                if (gi * kPair + kPair - 1 <= lim_min)
                    attend<NQ, kTwo, false>(st, gi == gw, q, img, gi * kPair, n, lim, p.scale_log2, lane);
                else
                    attend<NQ, kTwo, true>(st, gi == gw, q, img, gi * kPair, n, lim, p.scale_log2, lane);
                __syncwarp();
                if (lane == 0 && gi + kStages * step < g1) fetch(gi + kStages * step, stage);
                if (++stage == kStages) {
                    stage = 0;
                    parity ^= 1u;
                }
            }
            // ---- the warps' partials, in shared memory (every copy has been used)
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        so[(warp * R + 8 * i + 2 * cl + (e & 1)) * kRowPad + 16 * j + g + 8 * (e >> 1)] = st.o[j][i][e];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) st.l[i][e] += __shfl_xor_sync(0xffffffffu, st.l[i][e], x);
                    if (g == 0)
                        s_ml[warp][8 * i + 2 * cl + e] = make_float2(st.l[i][e] == 0.0f ? kLow : st.m[i][e], st.l[i][e]);
                }
            }
            if (cs > 1)
                cluster_sync();
            else
                __syncthreads();
            // ---- joined: rank x of the cluster has rows x, x + cs, ..; a warp joins the
            // partials that one CTA holds of one of them, then (cs > 1) the CTAs'
            auto write_row = [&](int r, int d, float4 o, float l) {
                const float inv = l > 0.0f ? 1.0f / l : l != l ? l : 0.0f;
                const int x = r / p.group, a = r - x * p.group;
                const int64_t at = (((int64_t)b * p.H * p.group + h * p.group + a) * p.t + x) * kD + d;
                if (p.out_dtype)
                    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
                else
                    *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + at) =
                        make_uint2(pack_h2(o.x * inv, o.y * inv), pack_h2(o.z * inv, o.w * inv));
            };
            const bool whole = start >= lo && unit_end <= hi;
            const int64_t slot = 2 * (int64_t)k + (start > lo ? 1 : 0);
            auto leave = [&](int r, int d, float m, float4 o, float l) {
                if (whole) {
                    write_row(r, d, o, l);
                } else {
                    *reinterpret_cast<float4*>(p.part_o + (slot * R + r) * kD + d) = o;
                    if (d == 0) p.part_ml[slot * R + r] = make_float2(m, l);
                }
            };
            const int mine = (rows - rank + cs - 1) / cs;  // this rank's rows
            for (int it = warp; it < mine * cs; it += kWarps) {
                const int r = rank + it / cs * cs, from = it % cs;
                float2 ml[kWarps];
                float4 v[kWarps];
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const uint32_t am = smem_u32(&s_ml[w][r]), ao = smem_u32(so + (w * R + r) * kRowPad + 4 * lane);
                    ml[w] = ld_cluster_v2(cs > 1 ? map_rank(am, from) : am);
                    v[w] = ld_cluster_v4(cs > 1 ? map_rank(ao, from) : ao);
                }
                float m = kLow, l = 0.0f;
                float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml[w].x);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = ex2(ml[w].x - m);
                    l += f * ml[w].y;
                    o.x += f * v[w].x, o.y += f * v[w].y, o.z += f * v[w].z, o.w += f * v[w].w;
                }
                if (cs == 1) {
                    leave(r, 4 * lane, m, o, l);
                } else {
                    *reinterpret_cast<float4*>(&s_part[it][4 * lane]) = o;
                    if (lane == 0) s_part_ml[it] = make_float2(m, l);
                }
            }
            // s_part[x count ..] (count <= 8), the partials of the rank's row x, joined by all
            // warps: 16 dims a warp, a partial for four lanes
            auto join = [&](int count, auto&& done) {
                const int share = lane >> 2;
                for (int it = warp; it < mine * 8; it += kWarps) {
                    const int x = it >> 3, d = 16 * (it & 7) + 4 * (lane & 3);
                    float2 ml = make_float2(kLow, 0.0f);
                    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (share < count) {
                        ml = s_part_ml[x * count + share];
                        o = *reinterpret_cast<const float4*>(&s_part[x * count + share][d]);
                    }
                    float m = ml.x;
#pragma unroll
                    for (int y = 4; y < 32; y <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, y));
                    const float f = ex2(ml.x - m);
                    float l = f * ml.y;
                    o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
                    for (int y = 4; y < 32; y <<= 1) {
                        l += __shfl_xor_sync(0xffffffffu, l, y);
                        o.x += __shfl_xor_sync(0xffffffffu, o.x, y);
                        o.y += __shfl_xor_sync(0xffffffffu, o.y, y);
                        o.z += __shfl_xor_sync(0xffffffffu, o.z, y);
                        o.w += __shfl_xor_sync(0xffffffffu, o.w, y);
                    }
                    if (share == 0) done(rank + x * cs, d, m, o, l);
                }
            };
            if (cs > 1) {
                __syncthreads();
                join(cs, leave);
            }
            if (!whole) {
                // ---- the last cluster to arrive joins the unit's partials (a rank its rows)
                const int k0 = start / sh.per, k1 = (unit_end - 1) / sh.per;
                __syncthreads();
                if (tid == 0) {
                    __threadfence();  // (the CTA's writes, which the barrier ordered before)
                    uint32_t* count = p.counters + k0 * 8 + rank;
                    s_last = atomicAdd(count, 1u) == (uint32_t)(k1 - k0);
                    if (s_last) *count = 0;
                    __threadfence();
                }
                __syncthreads();
                if (s_last) {
                    // `each` warps a row, every one a share of the clusters
                    const int each = max(1, kWarps / max(mine, 1));
                    for (int it = warp; it < mine * each; it += kWarps) {
                        const int r = rank + it / each * cs;
                        float m = kLow, l = 0.0f;
                        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        for (int x0 = k0 + it % each; x0 <= k1; x0 += 8 * each) {
                            float2 ml[8];
                            float4 v[8];
#pragma unroll
                            for (int y = 0; y < 8; ++y) {
                                const int x = x0 + y * each;
                                ml[y] = make_float2(kLow, 0.0f);
                                v[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                                if (x <= k1) {
                                    const int64_t at = (2 * (int64_t)x + (start > x * sh.per ? 1 : 0)) * R + r;
                                    ml[y] = __ldcg(&p.part_ml[at]);
                                    v[y] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * kD + 4 * lane));
                                }
                            }
                            float top = m;
#pragma unroll
                            for (int y = 0; y < 8; ++y) top = fmaxf(top, ml[y].x);
                            const float f0 = ex2(m - top);
                            m = top;
                            l *= f0;
                            o.x *= f0, o.y *= f0, o.z *= f0, o.w *= f0;
#pragma unroll
                            for (int y = 0; y < 8; ++y) {
                                const float f = ex2(ml[y].x - m);
                                l += f * ml[y].y;
                                o.x += f * v[y].x, o.y += f * v[y].y, o.z += f * v[y].z, o.w += f * v[y].w;
                            }
                        }
                        if (each == 1) {
                            write_row(r, 4 * lane, o, l);
                        } else {
                            *reinterpret_cast<float4*>(&s_part[it][4 * lane]) = o;
                            if (lane == 0) s_part_ml[it] = make_float2(m, l);
                        }
                    }
                    if (each > 1) {
                        __syncthreads();
                        join(each, [&](int r, int d, float, float4 o, float l) { write_row(r, d, o, l); });
                    }
                }
            }
            // (the ring's memory goes back to the copies)
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            if (cs > 1)
                cluster_sync();  // what other ranks read of this CTA is free, and nobody leaves before
            else
                __syncthreads();  // s_q, the merge area and s_last are free again
        }
        // ---- the next unit
        start = next_start;
        if (start < hi && ++h == p.H) {
            h = 0;
            n = seq_len(++b);
        }
    }
}

int row_tiles(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

constexpr int kMaxClusters = 2 * 152;  // two CTAs a SM, no clusters
constexpr size_t kCounterBytes = (size_t)kMaxClusters * 8 * 4;

size_t one_pass_bytes(int64_t rows) { return (size_t)2 * kMaxClusters * 8 * row_tiles(rows) * (8 + 4 * kD); }

// Clusters of cs CTAs (1, 2, 4, 8) that the GPU holds at once.
template <int NQ, bool kTwo>
cudaError_t resident_clusters(int cs, const cudaLaunchConfig_t& cfg, int& n) {
    static std::mutex mu;
    static int known[64][4] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    int& at = known[dev][cs == 1 ? 0 : cs == 2 ? 1 : cs == 4 ? 2 : 3];
    if (!at) {
        cudaError_t e = cudaFuncSetAttribute(fp4_attn_kernel<NQ, kTwo>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<NQ>);
        if (e != cudaSuccess) return e;
        cudaLaunchAttribute shape;
        shape.id = cudaLaunchAttributeClusterDimension;
        shape.val.clusterDim.x = cs;
        shape.val.clusterDim.y = shape.val.clusterDim.z = 1;
        cudaLaunchConfig_t probe = cfg;
        probe.gridDim = dim3((unsigned)cs, 1, 1);
        probe.attrs = &shape;
        probe.numAttrs = 1;
        int most = 0;
        e = cudaOccupancyMaxActiveClusters(&most, fp4_attn_kernel<NQ, kTwo>, &probe);
        if (e != cudaSuccess) return e;
        if (most < 1) return cudaErrorInvalidConfiguration;
        at = std::min(most, kMaxClusters / cs);
    }
    n = at;
    return cudaSuccess;
}

template <int NQ, bool kTwo>
cudaError_t launch_one_pass(cudaStream_t s, AttnParams& p, int64_t units) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes<NQ>;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    // Few units: the largest clusters of which every unit can have two (they join
    // on the chip what would be partials in memory), and units in whole ranges.
    // Many: CTAs of their own.
    int cs = 8;
    for (;; cs >>= 1) {
        const cudaError_t e = resident_clusters<NQ, kTwo>(cs, cfg, p.clusters);
        if (e != cudaSuccess) return e;
        p.pad = 2 * units <= p.clusters;
        if (p.pad || cs == 1) break;
    }
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cs;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    // Few units: one of up to four pairs a warp stays in one cluster, as the join of
    // several through memory takes longer (2.8 us) than the pairs (0.6 us each).
    const int64_t unit_pairs = std::max<int64_t>(1, (p.max_len + kPair - 1) / kPair);
    p.least = (p.pad && unit_pairs <= 4 * cs * kWarps ? 4 : 1) * cs * kWarps;
    // (a unit more than the places need: the padded split counts on it)
    const int64_t most = units * unit_pairs;
    p.clusters = (int)std::min<int64_t>(p.clusters, (most + p.least - 1) / p.least + units);
    cfg.gridDim = dim3((unsigned)(p.clusters * cs), 1, 1);
    return cudaLaunchKernelEx(&cfg, fp4_attn_kernel<NQ, kTwo>, p);
}

}  // namespace

size_t fp4_attn_workspace_bytes(int H, int group, int batch, int t, int64_t max_len) {
    const int64_t heads = (int64_t)batch * H, rows = (int64_t)t * group;
    const size_t few = one_pass_bytes(std::min<int64_t>(rows, kFp4Rows));
    return kCounterBytes + std::max(few, rows > kFp4RowsLeast ? fp4_tiles_workspace_bytes(heads, rows, max_len) : 0);
}

cudaError_t launch_fp4_attn(cudaStream_t s, const Fp4Attn& a) {
    const int64_t rows = (int64_t)a.t * a.group;
    // 17 to 32 rows: the tiles, while they are few (32 rows, in us, one pass and
    // tiles: 1 head of 16384 18.8 and 13.7, 8 heads of 8192 35 and 20, 2 heads of
    // 131072 45 and 38; 256 heads of 8192 175 and 231).  16 rows: 12.7 and 13.7,
    // 2 heads of 131072 28 and 37.
    const int64_t tiles = (int64_t)a.batch * a.map.H * ((std::min(a.max_len, a.cap) + 127) / 128);
    if (rows > kFp4Rows || (rows > kFp4RowsLeast && tiles <= 4096))
        return launch_fp4_tiles(s, a, static_cast<char*>(a.ws) + kCounterBytes);
    AttnParams p;
    p.rope = a.rope;
    p.q = a.q;
    p.map = a.map;
    p.seq_lens = a.seq_lens;
    p.max_len = (int)std::min(a.max_len, a.cap);
    p.batch = a.batch;
    p.t = a.t;
    p.group = a.group;
    p.H = a.map.H;
    p.out = a.out;
    p.out_dtype = a.out_dtype;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.status = a.status;
    const int nq = row_tiles(rows);
    char* ws = static_cast<char*>(a.ws);
    p.counters = reinterpret_cast<uint32_t*>(ws);
    p.part_o = reinterpret_cast<float*>(ws + kCounterBytes);
    p.part_ml = reinterpret_cast<float2*>(ws + kCounterBytes + (size_t)2 * kMaxClusters * 8 * nq * 4 * kD);
    const int64_t units = (int64_t)a.batch * a.map.H;
    switch (nq) {
        case 1: return a.out_dtype ? launch_one_pass<1, true>(s, p, units) : launch_one_pass<1, false>(s, p, units);
        case 2: return a.out_dtype ? launch_one_pass<2, true>(s, p, units) : launch_one_pass<2, false>(s, p, units);
        default: return a.out_dtype ? launch_one_pass<4, true>(s, p, units) : launch_one_pass<4, false>(s, p, units);
    }
}

}  // namespace bgtq
