// Attention of a few query rows over the 4-bit cache in one pass over its
// bytes (up to 32 rows of a KV head: a decode step of up to 8 query heads, or
// a few drafted tokens).
//
// out = sum_j softmax_j(scale q.k_j) v_j over the positions a row sees; split
// over the positions, one running maximum and sum per warp, partials joined by
// log-sum-exp.  A warp takes groups of 16 positions, brought to shared memory
// by bulk copies of 2304 bytes, kStages in flight a warp:
//   S^T = K Q^T   (16 positions x 8 rows, K 16 dims a step): codes to fp16 by
//                 the hardware's conversion, times the block's scale, exact;
//                 the products are fp16 x fp16 in fp32
//   P^T           exp2(scaled S - m) in fp32, split into two fp16 parts (22
//                 bits), transposed from accumulator to operand by movmatrix
//   O^T += V^T P^T  (16 dims x 8 rows, 16 positions a step), twice (two parts)
// A lane's operands are contiguous in a group (that is its layout), so a
// group is read with eight conflict-free loads a lane.  mma.sync, not tcgen05:
// 8 to 32 rows a head leave a 128-row tile idle, and its operands would have
// to pass through shared memory once more, decoded (4.5 -> 16 bits a value).
// The reference m of a row's exponentials stays kLift below the largest logit
// when set and moves only when a logit passes it by kRange, so that the two
// parts keep 22 bits well above fp16's smallest numbers.
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "fp4.cuh"
#include "tc_common.cuh"

namespace bgtq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 4;         // groups in flight a warp
constexpr int kRowPad = 132;       // floats of a row of partial output in shared memory (keeps the warp's stores on 32 banks)
constexpr float kLift = 8.0f, kRange = 15.0f;
constexpr float kLow = -1.0e30f;   // "no position yet"
constexpr int kMaxSlots = 152 * 16;  // partials of all units that a workspace has room for

struct AttnParams {
    RopeParams rope;
    RowsView q;
    Fp4Map map;
    const int32_t* seq_lens;
    int64_t cap, max_len;
    int t, group, H;
    int row_blocks;   // blocks of 8 NQ rows of a KV head's t * group; a unit is one of them
    int parts;        // splits of a unit (workspace slots)
    int part_groups;  // groups of a split
    void* out;
    int out_dtype;
    float scale_log2;
    uint32_t* counters;
    float2* part_ml;  // [slot][rows]: (m, l)
    float* part_o;    // [slot][rows][128]
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

// One group: img in shared memory, base its first position, lim the last
// position each of the lane's rows sees; kEdge: some position is not seen by
// every row (past n: its scales do not count).
template <int NQ, bool kEdge>
__device__ __forceinline__ void attend(State<NQ>& st, const uint32_t (&q)[8][NQ][2], const uint8_t* img, int base, int n,
                                       const int (&lim)[NQ][2], float c, int lane) {
    const int g = lane >> 2, cl = lane & 3;
    float s[NQ][4];
#pragma unroll
    for (int i = 0; i < NQ; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
    {
        const uint4 ka = *reinterpret_cast<const uint4*>(img + 64 * g + 16 * cl);
        const uint4 kb = *reinterpret_cast<const uint4*>(img + 64 * (g + 8) + 16 * cl);
        const uint2 sa = *reinterpret_cast<const uint2*>(img + kGroupKs + 8 * g);
        const uint2 sb = *reinterpret_cast<const uint2*>(img + kGroupKs + 8 * (g + 8));
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
                for (int i = 0; i < NQ; ++i) mma16816(s[i], a0, a1, a2, a3, q[2 * jj + k][i][0], q[2 * jj + k][i][1]);
            }
        }
    }
    // logits of positions g (0, 1) and g + 8 (2, 3), rows 2 cl (0, 2) and 2 cl + 1 (1, 3)
    bool over = false;
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[i][e] *= c;
            if (kEdge && base + g + 8 * (e >> 1) > lim[i][e & 1]) s[i][e] = -INFINITY;
            over |= s[i][e] > st.m[i][e & 1] + kRange;
        }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mt = fmaxf(s[i][e], s[i][e + 2]);
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
                if (mt > st.m[i][e] + kRange) {
                    const float f = ex2(st.m[i][e] - (mt - kLift));  // (0 the first time)
                    st.m[i][e] = mt - kLift;
                    st.l[i][e] *= f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        st.o[j][i][e] *= f;
                        st.o[j][i][e + 2] *= f;
                    }
                }
            }
    }
    uint32_t hi[NQ][2], lo[NQ][2];
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float p0 = ex2(s[i][2 * x] - st.m[i][0]), p1 = ex2(s[i][2 * x + 1] - st.m[i][1]);
            st.l[i][0] += p0;
            st.l[i][1] += p1;
            const __half2 h = __floats2half2_rn(p0, p1);
            const float2 b = __half22float2(h);
            hi[i][x] = transpose8(h2u(h));
            lo[i][x] = transpose8(h2u(__floats2half2_rn(p0 - b.x, p1 - b.y)));
        }
    uint32_t dead = 0xffffffffu;  // scale bytes of positions past the sequence: their bits do not count
    if (kEdge) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (base + 2 * cl + (e & 1) + 8 * (e >> 1) >= n) dead &= ~(0xffu << (8 * e));
    }
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
        const uint4 v = *reinterpret_cast<const uint4*>(img + kGroupV + 512 * jj + 16 * lane);
        const uint4 t = *reinterpret_cast<const uint4*>(img + kGroupVs + 32 * cl + 16 * jj);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w}, sc[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t u = kEdge ? sc[k] & dead : sc[k];
            const __half2 f0 = fp4_scales<0>(u), f1 = fp4_scales<2>(u);
            __half2 x[4];
            fp4_numbers(w[k], x);
            const uint32_t a0 = h2u(__hmul2(x[0], f0)), a1 = h2u(__hmul2(x[1], f0));
            const uint32_t a2 = h2u(__hmul2(x[2], f1)), a3 = h2u(__hmul2(x[3], f1));
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                mma16816(st.o[4 * jj + k][i], a0, a1, a2, a3, hi[i][0], hi[i][1]);
                mma16816(st.o[4 * jj + k][i], a0, a1, a2, a3, lo[i][0], lo[i][1]);
            }
        }
    }
}

template <int NQ>
constexpr int smem_ring() {
    return kWarps * kStages * kGroupBytes;
}
template <int NQ>
constexpr int smem_merge() {
    return kWarps * 8 * NQ * kRowPad * 4;
}
template <int NQ>
constexpr int smem_bytes() {
    return smem_ring<NQ>() > smem_merge<NQ>() ? smem_ring<NQ>() : smem_merge<NQ>();
}

template <int NQ>
__global__ void __launch_bounds__(kThreads, NQ == 1 ? 2 : 1) fp4_attn_kernel(const __grid_constant__ AttnParams p) {
    constexpr int R = 8 * NQ;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) __half s_q[R][kD + 8];
    __shared__ float s_m[kWarps][R], s_l[kWarps][R];
    __shared__ int s_lim[R];
    __shared__ __align__(8) uint64_t s_bar[kWarps * kStages];
    __shared__ int s_abort, s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int unit = blockIdx.x, part = blockIdx.y;
    const int head = unit / p.row_blocks, row0 = (unit - head * p.row_blocks) * R;
    const int b = head / p.H, h = head - b * p.H;
    const int rows = min(R, p.t * p.group - row0);  // of this unit
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid < kWarps * kStages) mbar_init(smem_u32(&s_bar[tid]), 1);
    if (tid == 0) s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int64_t n64 = p.seq_lens[b];
    if (n64 < 0 || n64 > p.max_len) {
        if (tid == 0 && part == 0 && h == 0 && p.status) atomicOr(p.status, BGTQ_STATUS_SEQLEN_CAPACITY);
        n64 = n64 < 0 ? 0 : p.max_len;
    }
    const int n = (int)n64;
    // groups that the unit's last row sees
    const int n_groups = (max(0, n - p.t + 1 + (row0 + rows - 1) / p.group) + kGroup - 1) / kGroup;
    const int active = max(1, (n_groups + p.part_groups - 1) / p.part_groups);  // splits that have positions
    if (part >= active) return;
    __syncthreads();  // barriers initialised
    const int g0 = part * p.part_groups, g1 = min(n_groups, g0 + p.part_groups);
    // ---- the warp's first groups
    uint8_t* ring = smem + warp * (kStages * kGroupBytes);
    const uint32_t ring_a = smem_u32(ring), bar_a = smem_u32(&s_bar[warp * kStages]);
    volatile int* abort_flag = &s_abort;
    auto fetch = [&](int gi, int stage) {
        const uint8_t* src = p.map.group(b, h, gi);
        if (!src) {
            if (p.status) atomicOr(p.status, BGTQ_STATUS_PAGE_RANGE);
            src = p.map.base;  // (some group of the pool: the output is unspecified)
        }
        mbar_expect_tx(bar_a + 8 * stage, kGroupBytes);
        bulk_copy(ring_a + stage * kGroupBytes, src, kGroupBytes, bar_a + 8 * stage);
    };
    if (lane == 0)
        for (int s = 0; s < kStages; ++s)
            if (g0 + warp + s * kWarps < g1) fetch(g0 + warp + s * kWarps, s);
    // ---- the query rows (row r: token r / group, query head h group + r mod group), rotated
    for (int r = warp; r < R; r += kWarps) {
        uint2 w = make_uint2(0u, 0u);
        int lim = n - 1;
        if (r < rows) {
            const int i = (row0 + r) / p.group, a = row0 + r - i * p.group;
            lim = n - p.t + i;
            const __half* row = static_cast<const __half*>(p.q.p) + b * p.q.sb + (int64_t)(h * p.group + a) * p.q.sh + i * p.q.st;
            if (p.rope.cos) {
                int pos[kMaxAxes];
                if (lim >= 0 && rope_positions(p.rope, (int64_t)b * p.t + i, lim, pos)) {
                    __half e[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) e[k] = rope_elem(p.rope, pos, row, 4 * lane + k);
                    w = make_uint2(__half_as_ushort(e[0]) | (uint32_t)__half_as_ushort(e[1]) << 16,
                                   __half_as_ushort(e[2]) | (uint32_t)__half_as_ushort(e[3]) << 16);
                } else {
                    if (lim >= 0 && lane == 0 && part == 0 && p.status) atomicOr(p.status, BGTQ_STATUS_ROPE_RANGE);
                    lim = -1;
                }
            } else {
                w = *reinterpret_cast<const uint2*>(row + 4 * lane);
            }
        }
        *reinterpret_cast<uint2*>(&s_q[r][4 * lane]) = w;
        if (lane == 0) s_lim[r] = lim;
    }
    __syncthreads();
    const int g = lane >> 2, cl = lane & 3;
    uint32_t q[8][NQ][2];
    int lim[NQ][2], lim_min = n - 1;
    State<NQ> st;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint2 w = *reinterpret_cast<const uint2*>(&s_q[8 * i + g][16 * j + 4 * cl]);
            q[j][i][0] = w.x;
            q[j][i][1] = w.y;
            st.o[j][i][0] = st.o[j][i][1] = st.o[j][i][2] = st.o[j][i][3] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            lim[i][e] = s_lim[8 * i + 2 * cl + e];
            lim_min = min(lim_min, lim[i][e]);
            st.m[i][e] = kLow;
            st.l[i][e] = 0.0f;
        }
    }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);
    // ---- the groups
    int stage = 0;
    uint32_t parity = 0;
    for (int gi = g0 + warp; gi < g1; gi += kWarps) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar_a + 8 * stage, parity, abort_flag, p.status))) {
            // gave up: the warp's own copies land (or time out once more) before the CTA ends
            for (int s = 0; s < kStages && gi + s * kWarps < g1; ++s) {
                mbar_wait(bar_a + 8 * stage, parity, abort_flag, p.status, false);
                if (++stage == kStages) {
                    stage = 0;
                    parity ^= 1u;
                }
            }
            break;
        }
        const uint8_t* img = ring + stage * kGroupBytes;
        if (gi * kGroup + kGroup - 1 <= lim_min)
            attend<NQ, false>(st, q, img, gi * kGroup, n, lim, p.scale_log2, lane);
        else
            attend<NQ, true>(st, q, img, gi * kGroup, n, lim, p.scale_log2, lane);
        __syncwarp();
        if (lane == 0 && gi + kStages * kWarps < g1) fetch(gi + kStages * kWarps, stage);
        if (++stage == kStages) {
            stage = 0;
            parity ^= 1u;
        }
    }
    // ---- the CTA's partial: the warps' joined in shared memory
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) st.l[i][e] += __shfl_xor_sync(0xffffffffu, st.l[i][e], x);
    __syncthreads();  // every warp is done with its ring
    if (s_abort) return;
    float* so = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                so[(warp * R + 8 * i + 2 * cl + (e & 1)) * kRowPad + 16 * j + g + 8 * (e >> 1)] = st.o[j][i][e];
        if (g == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s_m[warp][8 * i + 2 * cl + e] = st.m[i][e];
                s_l[warp][8 * i + 2 * cl + e] = st.l[i][e];
            }
        }
    }
    __syncthreads();
    auto write_row = [&](int r, float4 o, float l) {
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        const int i = (row0 + r) / p.group, a = row0 + r - i * p.group;
        const int64_t at = (((int64_t)b * p.H * p.group + h * p.group + a) * p.t + i) * kD + 4 * lane;
        if (p.out_dtype)
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        else
            *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + at) =
                make_uint2(pack_h2(o.x * inv, o.y * inv), pack_h2(o.z * inv, o.w * inv));
    };
    const int64_t slot0 = (int64_t)unit * p.parts;
    for (int r = warp; r < rows; r += kWarps) {
        float m = kLow, l = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_m[w][r]);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(s_m[w][r] - m);
            l += f * s_l[w][r];
            const float4 x = *reinterpret_cast<const float4*>(so + (w * R + r) * kRowPad + 4 * lane);
            o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
        }
        if (active == 1) {
            write_row(r, o, l);
        } else {
            *reinterpret_cast<float4*>(p.part_o + ((slot0 + part) * R + r) * kD + 4 * lane) = o;
            if (lane == 0) p.part_ml[(slot0 + part) * R + r] = make_float2(m, l);
        }
    }
    if (active == 1) return;
    // ---- the unit's last CTA joins the partials
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        const uint32_t before = atomicAdd(p.counters + unit, 1u);
        s_last = before + 1 == (uint32_t)active;
        if (s_last) p.counters[unit] = 0;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    for (int r = warp; r < rows; r += kWarps) {
        float m = kLow;
        for (int x = lane; x < active; x += 32) m = fmaxf(m, __ldcg(&p.part_ml[(slot0 + x) * R + r]).x);
#pragma unroll
        for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        float l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int x = 0; x < active; ++x) {
            const float2 ml = __ldcg(&p.part_ml[(slot0 + x) * R + r]);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part_o + ((slot0 + x) * R + r) * kD + 4 * lane));
            const float f = ex2(ml.x - m);
            l += f * ml.y;
            o.x += f * v.x, o.y += f * v.y, o.z += f * v.z, o.w += f * v.w;
        }
        write_row(r, o, l);
    }
}

// How a unit's positions are split.
struct Split {
    int parts, part_groups;
};
Split split_for(int64_t units, int64_t max_len) {
    const int64_t groups = std::max<int64_t>(1, (max_len + kGroup - 1) / kGroup);
    // one wave of two CTAs a SM where the units are few; about eight splits'
    // worth of CTAs a SM slot, of ragged sequences, where they are many
    const int64_t want = units < 152 ? std::max<int64_t>(1, 2 * 152 / units) : std::max<int64_t>(1, kMaxSlots / units);
    int64_t per = (groups + want - 1) / want;
    per = std::max<int64_t>(per, units < 152 ? kWarps : 8 * kWarps);
    per = (per + kWarps - 1) / kWarps * kWarps;
    return {(int)((groups + per - 1) / per), (int)per};
}

int row_tiles(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }
int64_t row_blocks(int64_t rows) { return (rows + 31) / 32; }

constexpr size_t kCounterBytes = (size_t)kMaxSlots * 4;  // a unit that is split has two slots at least

size_t one_pass_bytes(int64_t heads, int64_t rows, int64_t max_len) {
    const int64_t units = heads * row_blocks(rows);
    const int64_t groups = std::max<int64_t>(1, (max_len + kGroup - 1) / kGroup);
    const int64_t slots = std::min<int64_t>(kMaxSlots, units * ((groups + kWarps - 1) / kWarps));
    return (size_t)slots * 8 * row_tiles(rows) * (8 + 4 * kD);
}

template <int NQ>
cudaError_t launch_one_pass(cudaStream_t s, AttnParams& p, int64_t units) {
    static std::mutex mu;
    static bool done[64] = {false};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!done[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(fp4_attn_kernel<NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<NQ>());
            if (e != cudaSuccess) return e;
            done[dev] = true;
        }
    }
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)units, (unsigned)p.parts, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes<NQ>();
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fp4_attn_kernel<NQ>, p);
}

}  // namespace

size_t fp4_attn_workspace_bytes(int H, int group, int batch, int t, int64_t max_len) {
    const int64_t heads = (int64_t)batch * H, rows = (int64_t)t * group;
    const size_t few = one_pass_bytes(heads, std::min<int64_t>(rows, kFp4Rows), max_len);
    return kCounterBytes + std::max(few, rows > kFp4Rows ? fp4_tiles_workspace_bytes(heads, rows, max_len) : 0);
}

cudaError_t launch_fp4_attn(cudaStream_t s, const Fp4Attn& a) {
    const int64_t rows = (int64_t)a.t * a.group;
    if (rows > kFp4Rows) return launch_fp4_tiles(s, a, static_cast<char*>(a.ws) + kCounterBytes);
    const int64_t units = (int64_t)a.batch * a.map.H * row_blocks(rows);
    const Split sp = split_for(units, std::min(a.max_len, a.cap));
    AttnParams p;
    p.rope = a.rope;
    p.q = a.q;
    p.map = a.map;
    p.seq_lens = a.seq_lens;
    p.cap = a.cap;
    p.max_len = std::min(a.max_len, a.cap);
    p.t = a.t;
    p.group = a.group;
    p.H = a.map.H;
    p.parts = sp.parts;
    p.part_groups = sp.part_groups;
    p.out = a.out;
    p.out_dtype = a.out_dtype;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.status = a.status;
    p.row_blocks = (int)row_blocks(rows);
    const int nq = row_tiles(rows);
    char* ws = static_cast<char*>(a.ws);
    const int64_t slots = std::min<int64_t>(kMaxSlots, units * sp.parts);
    p.counters = reinterpret_cast<uint32_t*>(ws);
    p.part_o = reinterpret_cast<float*>(ws + kCounterBytes);
    p.part_ml = reinterpret_cast<float2*>(ws + kCounterBytes + (size_t)slots * 8 * nq * 4 * kD);
    switch (nq) {
        case 1: return launch_one_pass<1>(s, p, units);
        case 2: return launch_one_pass<2>(s, p, units);
        default: return launch_one_pass<4>(s, p, units);
    }
}

}  // namespace bgtq
