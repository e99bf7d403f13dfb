// Eviction from a packed cache by accumulated attention weight: of every
// (sequence, KV head) the first `sinks` and the last `recent` positions and,
// of the positions between, those of the largest score are kept, `keep` in
// all, and their records moved in position order into another packed cache.
//
// Two launches.  evict_select_kernel: one thread-block cluster per (sequence,
// KV head), each CTA with a contiguous segment of the positions, each warp
// with a contiguous part of it, the scores in registers as integers of the
// same order.  The threshold (the score that the last kept position has) is
// found by an exact radix selection: three histograms of 11, 11 and 10 bits
// from the top, each summed over the cluster through distributed shared
// memory between two cluster barriers; a seventh one joins the counts of what
// is kept.  Equal scores at the threshold are
// taken from the lowest position.  Every CTA then counts its share, and its
// warps write their positions at the index that the counts before them give:
// no atomics on global memory, the same result on every run.  The kernel is
// latency-bound (a few round trips per histogram), so a long sequence is
// spread over up to 16 CTAs and every loop over a thread's keys is unrolled.
// evict_move_kernel: 128 destination tokens per block; K records and norms
// are copies; a V record holds two tokens' codes in alternating bit fields,
// so each of its words is the even fields of one source word (shifted down by
// one field if the token sat in the odd half) joined with the odd fields of
// another.
#include <cooperative_groups.h>

#include <algorithm>
#include <mutex>

#include "bgtq_internal.h"

namespace bgtq {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kSelMaxCluster = 16;
constexpr int kMoveThreads = 256;
constexpr int kMoveTok = 128;        // destination tokens of a block (even)
constexpr int kMoveBatch = 2;        // record pieces of a thread in flight (1: 19.1 us for 128K -> 32K, 2: 18.7, 3: 18.4; for 32 x 8 units 63, 64, 72 us)

__device__ __forceinline__ void evict_pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void evict_pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct EvictParams {
    const float* scores;  // [B][H][cap]
    int64_t cap;
    const int32_t* seq_lens;
    int64_t max_len;      // longer sequences are cut to it (flagged)
    int keep, sinks, recent;
    int32_t* kept;        // [B][H][keep] source positions, ascending; -1 past the kept ones
    float* dst_scores;    // [B][H][dst_cap]
    int64_t dst_cap;
    int32_t* dst_lens;    // [B]
    const uint8_t* kc;
    const float* kn;
    const uint8_t* vc;
    const float* vn;
    CacheMap map;
    uint8_t* dkc;
    float* dkn;
    uint8_t* dvc;
    float* dvn;
    CacheMap dmap;
    int H, bk;
    int32_t* status;
};

// Length of sequence b, cut to what the cache and the call allow (read by the
// selection alone, after its wait).
__device__ __forceinline__ int evict_len(const EvictParams& p, int b, bool report) {
    const int n = p.seq_lens[b];
    const int64_t lim = min(p.cap, p.max_len);
    if (n >= 0 && n <= lim) return n;
    if (report && p.status) atomicOr(p.status, BGTQ_STATUS_SEQLEN_CAPACITY);
    return n < 0 ? 0 : (int)lim;
}

// Integers in the order of the scores: -0 and +0 are one value, NaN the lowest.
__device__ __forceinline__ uint32_t score_key(float f) {
    if (f != f) return 0u;
    const uint32_t u = f == 0.0f ? 0u : __float_as_uint(f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

struct __align__(16) SelShared {
    uint32_t hist[3][kSelBins];
    uint32_t total[kSelBins];  // the cluster's histogram
    uint32_t warp_sum[kSelWarps];
    uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
    uint32_t cta_gt, cta_eq;
    uint32_t bin, above;
};

// KPT: keys per thread (8, 16 or 32; 32 KPT positions per warp), or 0: any
// number, read from global memory on every pass.
template <int KPT>
__global__ void __launch_bounds__(kSelThreads, KPT > 16 ? 1 : 2) evict_select_kernel(EvictParams p) {
    __shared__ SelShared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int crank = (int)cluster.block_rank(), csize = (int)cluster.num_blocks();
    const int h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const size_t unit = (size_t)b * p.H + h;
    // (with nothing to move no kernel of this call follows, and the lengths
    // written here may be what the next one reads before it waits)
    if (p.max_len > 0) evict_pdl_trigger();
    for (int i = tid; i < 3 * kSelBins / 4; i += kSelThreads) reinterpret_cast<uint4*>(&s.hist[0][0])[i] = make_uint4(0, 0, 0, 0);
    evict_pdl_wait();
    const int n = evict_len(p, b, h == 0 && crank == 0 && tid == 0);
    const int m = min(n, p.keep);
    int32_t* kept = p.kept + unit * (size_t)p.keep;
    if (h == 0 && crank == 0 && tid == 0) p.dst_lens[b] = m;
    for (int64_t i = (int64_t)m + crank * kSelThreads + tid; i < p.keep; i += csize * kSelThreads) kept[i] = -1;
    if (n <= p.keep) {  // everything stays (the whole cluster leaves here)
        for (int i = crank * kSelThreads + tid; i < n; i += csize * kSelThreads) kept[i] = i;
        return;
    }
    // candidates [c0, c1); the positions outside always stay
    const int c0 = p.sinks, c1 = n - p.recent;  // n > keep >= sinks + recent
    uint32_t need = (uint32_t)(p.keep - p.sinks - p.recent);
    const bool none = need == 0;  // the sinks and the recent positions fill the budget
    // the warp's positions: groups of 32 from w0
    const int wn = KPT > 0 ? 32 * KPT : ((n + csize * kSelWarps - 1) / (csize * kSelWarps) + 31) & ~31;
    const int w0 = (int)min((int64_t)n, ((int64_t)crank * kSelWarps + warp) * wn), w1 = (int)min((int64_t)n, (int64_t)w0 + wn);
    const float* row = p.scores + unit * (size_t)p.cap;
    // keys of the lane's positions, and which of them are candidates (bit j)
    uint32_t key[KPT > 0 ? KPT : 1], cand = 0;
    if constexpr (KPT > 0) {
        float x[KPT];
#pragma unroll
        for (int j = 0; j < KPT; ++j) {
            const int i = w0 + 32 * j + lane;
            x[j] = i < w1 ? __ldg(row + i) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < KPT; ++j) {
            const int i = w0 + 32 * j + lane;
            key[j] = score_key(x[j]);
            cand |= (i < w1 && i >= c0 && i < c1 ? 1u : 0u) << j;
        }
    }
    // f(position, key, whether it is a candidate) for every group of 32
    // positions of the warp, in order
    auto groups = [&](auto&& f) {
        if constexpr (KPT > 0) {
#pragma unroll
            for (int j = 0; j < KPT; ++j) f(w0 + 32 * j + lane, key[j], ((cand >> j) & 1u) != 0);
        } else {
            for (int i0 = w0; i0 < w1; i0 += 32) {
                const int i = i0 + lane;
                f(i, i < w1 ? score_key(__ldg(row + i)) : 0u, i < w1 && i >= c0 && i < c1);
            }
        }
    };
    __syncthreads();  // the histograms are zero

    uint32_t prefix = 0;  // the threshold's bits found so far
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        if (none) break;
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 2 ? 1023u : 2047u;
        uint32_t* hist = s.hist[pass];
        groups([&](int, uint32_t k, bool in) {
            if (in && (pass == 0 || (pass == 1 ? (k >> 21) == prefix : (k >> 10) == prefix)))
                atomicAdd(hist + ((k >> shift) & mask), 1u);
        });
        // the cluster's histogram: CTA r sums a share of the bins over the
        // cluster and writes it to every CTA (all bins read by every CTA
        // would be csize times the traffic between the SMs)
        const uint32_t* total = hist;
        if (csize > 1) {
            cluster.sync();
            total = s.total;
            const int share = kSelBins / csize, b0 = crank * share;  // (csize: a power of two)
            for (int q = tid; q < share; q += kSelThreads) {
                uint32_t r[kSelMaxCluster], sum = 0;
#pragma unroll
                for (int c = 0; c < kSelMaxCluster; ++c)
                    r[c] = c < csize ? *cluster.map_shared_rank(hist + b0 + q, c) : 0u;
#pragma unroll
                for (int c = 0; c < kSelMaxCluster; ++c) sum += r[c];
#pragma unroll
                for (int c = 0; c < kSelMaxCluster; ++c)
                    if (c < csize) *cluster.map_shared_rank(s.total + b0 + q, c) = sum;
            }
            cluster.sync();
        } else {
            __syncthreads();
        }
        // four bins a thread, from the top
        static_assert(kSelBins == 4 * kSelThreads, "16-byte reads of four bins");
        const int hb = kSelBins - 4 * (tid + 1);
        const uint4 v = *reinterpret_cast<const uint4*>(total + hb);
        uint32_t inc = (v.x + v.y) + (v.z + v.w);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += x;
        }
        if (lane == 31) s.warp_sum[warp] = inc;
        __syncthreads();
        const uint32_t before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? s.warp_sum[lane] : 0u);
        // candidates above bin hb + 3, hb + 2, hb + 1, hb; the bin that the
        // need-th falls into
        const uint32_t a3 = before + inc - ((v.x + v.y) + (v.z + v.w)), a2 = a3 + v.w, a1 = a2 + v.z, a0 = a1 + v.y;
        if (a3 < need && need <= a0 + v.x) {
            s.bin = (uint32_t)hb + (need <= a2 ? 3u : need <= a1 ? 2u : need <= a0 ? 1u : 0u);
            s.above = need <= a2 ? a3 : need <= a1 ? a2 : need <= a0 ? a1 : a0;
        }
        __syncthreads();
        prefix = pass == 2 ? (prefix << 10) | s.bin : (prefix << 11) | s.bin;
        need -= s.above;
        // (warp_sum, bin, above and total are written again only after the
        // next pass's first barrier)
    }
    // threshold: candidates above `prefix` and the first `need` equal to it stay
    uint32_t gt = 0, eq = 0;
    groups([&](int, uint32_t k, bool in) {
        gt += in && !none && k > prefix ? 1u : 0u;
        eq += in && !none && k == prefix ? 1u : 0u;
    });
    gt = __reduce_add_sync(0xFFFFFFFFu, gt);
    eq = __reduce_add_sync(0xFFFFFFFFu, eq);
    if (lane == 0) {
        s.warp_gt[warp] = gt;
        s.warp_eq[warp] = eq;
    }
    __syncthreads();
    // candidates before the warp's positions: of its CTA's earlier warps, and
    // of the cluster's earlier CTAs
    uint32_t gb = lane < kSelWarps ? s.warp_gt[lane] : 0u, eb = lane < kSelWarps ? s.warp_eq[lane] : 0u;
    if (warp == 0) {
        const uint32_t g = __reduce_add_sync(0xFFFFFFFFu, gb), e = __reduce_add_sync(0xFFFFFFFFu, eb);
        if (lane == 0) {
            s.cta_gt = g;
            s.cta_eq = e;
        }
    }
    cluster.sync();
    if (lane >= warp) gb = eb = 0u;
    if (lane < crank) {
        gb += *cluster.map_shared_rank(&s.cta_gt, lane);
        eb += *cluster.map_shared_rank(&s.cta_eq, lane);
    }
    gb = __reduce_add_sync(0xFFFFFFFFu, gb);
    eb = __reduce_add_sync(0xFFFFFFFFu, eb);
    // (no CTA leaves while another may read its counts)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    // kept positions before the warp's: the ones that always stay among the
    // w0 first positions, the candidates above the threshold, the equal ones
    uint32_t at = (uint32_t)(min(w0, c0) + max(0, w0 - c1)) + gb + min(eb, need);
    const uint32_t lt = (1u << lane) - 1u;
    groups([&](int i, uint32_t k, bool in) {
        bool stays = i < w1 && (!in || (!none && k > prefix));
        const uint32_t be = __ballot_sync(0xFFFFFFFFu, in && !none && k == prefix);
        if (be != 0) {
            if (in && !none && k == prefix) stays = eb + (uint32_t)__popc(be & lt) < need;
            eb += (uint32_t)__popc(be);
        }
        const uint32_t bs = __ballot_sync(0xFFFFFFFFu, stays);
        if (stays) kept[at + (uint32_t)__popc(bs & lt)] = i;
        at += (uint32_t)__popc(bs);
    });
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Bits of the even tokens' fields in word w of a V record: bit i belongs to
// them when (32 w + i) mod 2 bV < bV.
template <int BV>
__device__ __forceinline__ uint32_t even_fields(int w) {
    uint32_t mask = 0;
    const int at = (32 * w) % (2 * BV);
#pragma unroll
    for (int i = 0; i < 32; ++i) mask |= ((at + i) % (2 * BV) < BV ? 1u : 0u) << i;
    return mask;
}

template <int BV>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictParams p) {
    __shared__ int64_t s_src[kMoveTok];  // source record slot of each token
    __shared__ int64_t s_dst[kMoveTok];  // destination record slot (-1: not written)
    __shared__ int s_pos[kMoveTok];
    __shared__ __align__(16) uint32_t s_even[8 * BV];
    // No early start of the next kernel from here: it may be a decode, which
    // reads its lengths before it waits, and those may be dst_lens.
    const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const size_t unit = (size_t)b * p.H + h;
    if (tid < 8 * BV) s_even[tid] = even_fields<BV>(tid);
    evict_pdl_wait();
    // The kept count is the one that the selection wrote, read after the wait:
    // seq_lens may come from a kernel that is still running when this one
    // starts, and another count than the selection's would take the -1 past
    // the kept positions for positions.  (At most as many as `kept` holds.)
    const int m = min(p.dst_lens[b], (int)min((int64_t)p.keep, min(p.cap, p.max_len)));
    const int d0 = blockIdx.x * kMoveTok;
    const int nt = min(kMoveTok, m - d0);
    if (nt <= 0) return;
    for (int i = tid; i < nt; i += kMoveThreads) {
        int pos = p.kept[unit * (size_t)p.keep + d0 + i];
        int64_t dst = p.dmap.slot(b, h, d0 + i);
        if (dst < 0 && p.status) atomicOr(p.status, BGTQ_STATUS_PAGE_RANGE);
        if (pos < 0 || pos >= min(p.cap, p.max_len)) {
            // not the selection's: a call on another stream has written to
            // this call's `kept` (nothing is read or moved by it)
            if (p.status) atomicOr(p.status, BGTQ_STATUS_SEQLEN_CAPACITY);
            pos = 0;
            dst = -1;
        }
        int64_t src = p.map.slot(b, h, pos);
        if (src < 0 && p.status) atomicOr(p.status, BGTQ_STATUS_PAGE_RANGE);
        if (src < 0) src = (int64_t)h << p.map.lp | (pos & ((1 << p.map.lp) - 1));  // an unmapped page: page 0 is read
        s_src[i] = src;
        s_dst[i] = dst;
        s_pos[i] = pos;
    }
    __syncthreads();
    // (all of a step's loads before its stores: the compiler may not move a
    // load over a store that could overlap it)
    for (int i = tid; i < nt; i += kMoveThreads) {
        const float sc = __ldg(p.scores + unit * (size_t)p.cap + s_pos[i]), kn = __ldg(p.kn + s_src[i]), vn = __ldg(p.vn + s_src[i]);
        p.dst_scores[unit * (size_t)p.dst_cap + d0 + i] = sc;
        if (s_dst[i] >= 0) {
            p.dkn[s_dst[i]] = kn;
            p.dvn[s_dst[i]] = vn;
        }
    }
    // 16-byte pieces, kMoveBatch a thread at a time: the K records' pieces,
    // then the V records'.  A V piece joins the even fields of one source with
    // the odd ones of the other (of a single last token: the record's own odd
    // fields stay).
    const uint4* ksrc = reinterpret_cast<const uint4*>(p.kc);
    uint4* kdst = reinterpret_cast<uint4*>(p.dkc);
    const uint32_t* vsrc = reinterpret_cast<const uint32_t*>(p.vc);
    uint32_t* vdst = reinterpret_cast<uint32_t*>(p.dvc);
    constexpr int kW = 8 * BV, kPieces = 2 * BV;
    const int nk = nt * p.bk, n = nk + (nt + 1) / 2 * kPieces;
    for (int i0 = tid; i0 < n; i0 += kMoveBatch * kMoveThreads) {
        uint4 x[kMoveBatch], y[kMoveBatch];
        uint32_t up[kMoveBatch], down[kMoveBatch];
#pragma unroll
        for (int u = 0; u < kMoveBatch; ++u) {
            const int i = i0 + u * kMoveThreads;
            if (i < nk) {
                const int t = i / p.bk;
                x[u] = __ldg(ksrc + s_src[t] * p.bk + (i - t * p.bk));
            } else if (i < n) {
                const int pr = (i - nk) / kPieces, w = 4 * (i - nk - pr * kPieces);
                const uint32_t* ra = vsrc + (s_src[2 * pr] >> 1) * kW + w;
                x[u] = __ldg(reinterpret_cast<const uint4*>(ra));
                up[u] = w + 4 < kW ? __ldg(ra + 4) : 0u;
                if (2 * pr + 1 < nt) {
                    const uint32_t* rb = vsrc + (s_src[2 * pr + 1] >> 1) * kW + w;
                    y[u] = __ldg(reinterpret_cast<const uint4*>(rb));
                    down[u] = w > 0 ? __ldg(rb - 1) : 0u;
                } else if (s_dst[2 * pr] >= 0) {
                    y[u] = *reinterpret_cast<const uint4*>(vdst + (s_dst[2 * pr] >> 1) * kW + w);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kMoveBatch; ++u) {
            const int i = i0 + u * kMoveThreads;
            if (i < nk) {
                const int t = i / p.bk;
                if (s_dst[t] >= 0) kdst[s_dst[t] * p.bk + (i - t * p.bk)] = x[u];
            } else if (i < n) {
                const int pr = (i - nk) / kPieces, w = 4 * (i - nk - pr * kPieces);
                const int64_t dst = s_dst[2 * pr];
                if (dst < 0) continue;
                uint4 a = x[u], b4 = y[u];
                if (s_src[2 * pr] & 1)  // an odd token's fields move down to the even ones
                    a = make_uint4(__funnelshift_r(a.x, a.y, BV), __funnelshift_r(a.y, a.z, BV), __funnelshift_r(a.z, a.w, BV),
                                   __funnelshift_r(a.w, up[u], BV));
                if (2 * pr + 1 < nt && !(s_src[2 * pr + 1] & 1))  // an even token's fields move up
                    b4 = make_uint4(__funnelshift_l(down[u], b4.x, BV), __funnelshift_l(b4.x, b4.y, BV),
                                    __funnelshift_l(b4.y, b4.z, BV), __funnelshift_l(b4.z, b4.w, BV));
                const uint4 e = *reinterpret_cast<const uint4*>(s_even + w);
                *reinterpret_cast<uint4*>(vdst + (dst >> 1) * kW + w) =
                    make_uint4((a.x & e.x) | (b4.x & ~e.x), (a.y & e.y) | (b4.y & ~e.y), (a.z & e.z) | (b4.z & ~e.z),
                               (a.w & e.w) | (b4.w & ~e.w));
            }
        }
    }
}

}  // namespace

cudaError_t launch_evict(const bgtq_plan& pl, cudaStream_t s, const bgtq_cache& src, const float* scores,
                         const int32_t* seq_lens, int64_t max_len, int batch, int keep, int sinks, int recent,
                         const bgtq_cache& dst, float* dst_scores, int32_t* dst_lens, int32_t* kept, int32_t* status) {
    static std::mutex mu;
    static bool done[64] = {false};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!done[dev]) {  // clusters of 16 CTAs
            constexpr cudaFuncAttribute kAttr = cudaFuncAttributeNonPortableClusterSizeAllowed;
            cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<0>, kAttr, 1);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(evict_select_kernel<8>, kAttr, 1);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(evict_select_kernel<16>, kAttr, 1);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(evict_select_kernel<32>, kAttr, 1);
            if (e != cudaSuccess) return e;
            done[dev] = true;
        }
    }
    EvictParams p;
    p.scores = scores;
    p.cap = src.capacity;
    p.seq_lens = seq_lens;
    p.max_len = max_len;
    p.keep = keep;
    p.sinks = sinks;
    p.recent = recent;
    p.kept = kept;
    p.dst_scores = dst_scores;
    p.dst_cap = dst.capacity;
    p.dst_lens = dst_lens;
    p.kc = static_cast<const uint8_t*>(src.k_codes);
    p.kn = src.k_norm;
    p.vc = static_cast<const uint8_t*>(src.v_codes);
    p.vn = src.v_norm;
    p.map = make_cache_map(src, pl.H, batch, status);
    p.dkc = static_cast<uint8_t*>(dst.k_codes);
    p.dkn = dst.k_norm;
    p.dvc = static_cast<uint8_t*>(dst.v_codes);
    p.dvn = dst.v_norm;
    p.dmap = make_cache_map(dst, pl.H, batch, status);
    p.H = pl.H;
    p.bk = pl.bk;
    p.status = status;
    // CTAs per unit: as few as hold its keys in registers, and more while they
    // leave SMs idle and a thread has over 8 keys (32 x 8 units of up to 16384
    // positions: 64 us with a CTA each, 74 with clusters of two)
    int csize = 1;
    const int64_t units = (int64_t)batch * pl.H, two_waves = 2 * (int64_t)std::max(1, pl.num_sms);
    auto keys = [&] { return (max_len + (int64_t)csize * kSelThreads - 1) / ((int64_t)csize * kSelThreads); };
    while (csize < kSelMaxCluster && (keys() > 32 || (units * csize * 2 <= two_waves && keys() > 8))) csize *= 2;
    const int64_t kpt = keys();
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)csize;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)csize, (unsigned)pl.H, (unsigned)batch);
    cfg.blockDim = dim3(kSelThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = kpt <= 8    ? cudaLaunchKernelEx(&cfg, evict_select_kernel<8>, p)
                    : kpt <= 16 ? cudaLaunchKernelEx(&cfg, evict_select_kernel<16>, p)
                    : kpt <= 32 ? cudaLaunchKernelEx(&cfg, evict_select_kernel<32>, p)
                                : cudaLaunchKernelEx(&cfg, evict_select_kernel<0>, p);
    if (e != cudaSuccess) return e;
    const int64_t most = std::min<int64_t>(keep, max_len);
    if (most == 0) return cudaSuccess;
    cudaLaunchConfig_t mv = {};
    mv.gridDim = dim3((unsigned)((most + kMoveTok - 1) / kMoveTok), (unsigned)pl.H, (unsigned)batch);
    mv.blockDim = dim3(kMoveThreads, 1, 1);
    mv.stream = s;
    mv.attrs = attr;
    mv.numAttrs = 1;
    switch (pl.bv) {
        case 1: return cudaLaunchKernelEx(&mv, evict_move_kernel<1>, p);
        case 2: return cudaLaunchKernelEx(&mv, evict_move_kernel<2>, p);
        case 3: return cudaLaunchKernelEx(&mv, evict_move_kernel<3>, p);
        case 4: return cudaLaunchKernelEx(&mv, evict_move_kernel<4>, p);
        case 5: return cudaLaunchKernelEx(&mv, evict_move_kernel<5>, p);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace bgtq
