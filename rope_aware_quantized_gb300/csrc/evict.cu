// Eviction from a packed cache by accumulated attention weight: of every
// (sequence, KV head) the first `sinks` and the last `recent` positions and,
// of the positions between, those of the largest score are kept, `keep` in
// all, and their records moved in position order into another packed cache.
//
// Two launches.  evict_select_kernel: one thread-block cluster per (sequence,
// KV head), each CTA with a contiguous segment of the positions, its scores
// in shared memory as integers of the same order.  The threshold (the score
// that the last kept position has) is found by an exact radix selection: three
// histograms of 11, 11 and 10 bits from the top, each summed over the cluster
// through distributed shared memory, one cluster barrier apiece.  Equal
// scores at the threshold are taken from the lowest position.  Every CTA then
// counts its share, and its warps write their positions at the index that the
// counts before them give: no atomics on global memory, the same result on
// every run.  evict_move_kernel: 128 destination tokens per block; K records
// and norms are copies; a V record holds two tokens' codes in alternating
// bit fields, so each of its words is the even fields of one source word
// (shifted down by one field if the token sat in the odd half) joined with
// the odd fields of another.
#include <cooperative_groups.h>

#include <algorithm>
#include <mutex>

#include "bgtq_internal.h"

namespace bgtq {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kSelKeys = 32768;      // scores of a segment kept in shared memory (128 KB); longer ones are read again
constexpr int kSelMaxCluster = 8;
constexpr int kSelPerCta = 4096;     // positions a CTA takes before the cluster grows
constexpr int kMoveThreads = 256;
constexpr int kMoveTok = 128;        // destination tokens of a block (even)

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

// Length of sequence b, cut to what the cache and the call allow.
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

struct SelShared {
    uint32_t hist[3][kSelBins];
    uint32_t warp_sum[kSelWarps];
    uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
    uint32_t cta_gt, cta_eq;
    uint32_t bin, above;
};

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(EvictParams p, int keys_in_smem) {
    extern __shared__ uint32_t s_key[];
    __shared__ SelShared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int crank = (int)cluster.block_rank(), csize = (int)cluster.num_blocks();
    const int h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const size_t unit = (size_t)b * p.H + h;
    evict_pdl_trigger();
    for (int i = tid; i < 3 * kSelBins; i += kSelThreads) (&s.hist[0][0])[i] = 0;
    evict_pdl_wait();
    const int n = evict_len(p, b, h == 0 && crank == 0 && tid == 0);
    const int m = min(n, p.keep);
    int32_t* kept = p.kept + unit * (size_t)p.keep;
    if (h == 0 && crank == 0 && tid == 0) p.dst_lens[b] = m;
    for (int i = m + crank * kSelThreads + tid; i < p.keep; i += csize * kSelThreads) kept[i] = -1;
    if (n <= p.keep) {  // everything stays (the whole cluster leaves here)
        for (int i = crank * kSelThreads + tid; i < n; i += csize * kSelThreads) kept[i] = i;
        return;
    }
    // candidates [c0, c1); the positions outside always stay
    const int c0 = p.sinks, c1 = n - p.recent;  // n > keep >= sinks + recent
    uint32_t need = (uint32_t)(p.keep - p.sinks - p.recent);
    const int seg = ((n + csize - 1) / csize + 31) & ~31;
    const int a0 = min(n, crank * seg), a1 = min(n, a0 + seg);
    const float* row = p.scores + unit * (size_t)p.cap;
    const bool in_smem = seg <= keys_in_smem;
    if (in_smem) {
        for (int i = a0 + tid; i < a1; i += kSelThreads) s_key[i - a0] = score_key(row[i]);
    }
    __syncthreads();
    auto key_at = [&](int i) -> uint32_t { return in_smem ? s_key[i - a0] : score_key(__ldg(row + i)); };

    uint32_t prefix = 0;  // the threshold's bits found so far
    for (int pass = 0; pass < 3 && need > 0; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 2 ? 1023u : 2047u;
        const int lo = max(a0, c0), hi = min(a1, c1);
        for (int i0 = lo; i0 < hi; i0 += kSelThreads) {
            const int i = i0 + tid;
            uint32_t digit = 0xFFFFFFFFu;
            if (i < hi) {
                const uint32_t k = key_at(i);
                const bool mine = pass == 0 || (pass == 1 ? (k >> 21) == prefix : (k >> 10) == prefix);
                if (mine) digit = (k >> shift) & mask;
            }
            // lanes with the same digit add once (equal scores would
            // serialise otherwise)
            const uint32_t peers = __match_any_sync(0xFFFFFFFFu, digit);
            if (digit != 0xFFFFFFFFu && lane == __ffs(peers) - 1) atomicAdd(&s.hist[pass][digit], (uint32_t)__popc(peers));
        }
        cluster.sync();
        // the cluster's histogram, two bins a thread from the top
        const int hb = kSelBins - 2 - 2 * tid;
        uint32_t v1 = 0, v0 = 0;  // bins hb + 1, hb
        for (int c = 0; c < csize; ++c) {
            const uint2 r = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&s.hist[pass][hb], c));
            v0 += r.x;
            v1 += r.y;
        }
        uint32_t inc = v0 + v1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += x;
        }
        if (lane == 31) s.warp_sum[warp] = inc;
        __syncthreads();
        uint32_t before = 0;
        for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
        const uint32_t above1 = before + inc - v0 - v1, above0 = above1 + v1;
        if (above1 < need && need <= above0) {
            s.bin = (uint32_t)hb + 1;
            s.above = above1;
        } else if (above0 < need && need <= above0 + v0) {
            s.bin = (uint32_t)hb;
            s.above = above0;
        }
        __syncthreads();
        prefix = pass == 2 ? (prefix << 10) | s.bin : (prefix << 11) | s.bin;
        need -= s.above;
        __syncthreads();  // warp_sum, bin and above are written again
    }
    // threshold: candidates above `prefix` and the first `need` equal to it
    // stay (none if the sinks and the recent positions fill the budget)
    const bool none = p.keep == p.sinks + p.recent;
    const int wseg = ((seg + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int w0 = min(a1, a0 + warp * wseg), w1 = min(a1, w0 + wseg);
    uint32_t gt = 0, eq = 0;
    if (!none) {
        for (int i0 = w0; i0 < w1; i0 += 32) {
            const int i = i0 + lane;
            const bool cand = i < w1 && i >= c0 && i < c1;
            const uint32_t k = cand ? key_at(i) : 0u;
            gt += (uint32_t)__popc(__ballot_sync(0xFFFFFFFFu, cand && k > prefix));
            eq += (uint32_t)__popc(__ballot_sync(0xFFFFFFFFu, cand && k == prefix));
        }
    }
    if (lane == 0) {
        s.warp_gt[warp] = gt;
        s.warp_eq[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t g = 0, e = 0;
        for (int w = 0; w < kSelWarps; ++w) {
            const uint32_t wg = s.warp_gt[w], we = s.warp_eq[w];
            s.warp_gt[w] = g;
            s.warp_eq[w] = e;
            g += wg;
            e += we;
        }
        s.cta_gt = g;
        s.cta_eq = e;
    }
    cluster.sync();
    uint32_t gb = s.warp_gt[warp], eb = s.warp_eq[warp];  // candidates before the warp's positions
    for (int c = 0; c < crank; ++c) {
        gb += *cluster.map_shared_rank(&s.cta_gt, c);
        eb += *cluster.map_shared_rank(&s.cta_eq, c);
    }
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const bool cand = i < w1 && i >= c0 && i < c1;
        const uint32_t k = cand && !none ? key_at(i) : 0u;
        const bool isg = cand && !none && k > prefix, ise = cand && !none && k == prefix;
        const uint32_t bg = __ballot_sync(0xFFFFFFFFu, isg), be = __ballot_sync(0xFFFFFFFFu, ise);
        const uint32_t lt = (1u << lane) - 1u;
        const uint32_t g = gb + (uint32_t)__popc(bg & lt), e = eb + (uint32_t)__popc(be & lt);
        const bool stays = i < w1 && (!cand || isg || (ise && e < need));
        if (stays) {
            const uint32_t always = (uint32_t)(min(i, c0) + max(0, i - c1));
            kept[always + g + min(e, need)] = i;
        }
        gb += (uint32_t)__popc(bg);
        eb += (uint32_t)__popc(be);
    }
    cluster.sync();  // no CTA leaves while another may read its counts
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
    __shared__ uint32_t s_even[8 * BV];
    const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const size_t unit = (size_t)b * p.H + h;
    evict_pdl_trigger();
    if (tid < 8 * BV) s_even[tid] = even_fields<BV>(tid);
    const int m = min(evict_len(p, b, false), p.keep);
    const int d0 = blockIdx.x * kMoveTok;
    const int nt = min(kMoveTok, m - d0);
    evict_pdl_wait();
    if (nt <= 0) return;
    for (int i = tid; i < nt; i += kMoveThreads) {
        const int pos = p.kept[unit * (size_t)p.keep + d0 + i];
        int64_t src = p.map.slot(b, h, pos);
        const int64_t dst = p.dmap.slot(b, h, d0 + i);
        if ((src < 0 || dst < 0) && p.status) atomicOr(p.status, BGTQ_STATUS_PAGE_RANGE);
        if (src < 0) src = (int64_t)h << p.map.lp | (pos & ((1 << p.map.lp) - 1));  // an unmapped page: page 0 is read
        s_src[i] = src;
        s_dst[i] = dst;
        p.dst_scores[unit * (size_t)p.dst_cap + d0 + i] = p.scores[unit * (size_t)p.cap + pos];
        if (dst >= 0) {
            p.dkn[dst] = p.kn[src];
            p.dvn[dst] = p.vn[src];
        }
    }
    __syncthreads();
    // K records, 16 bytes a step
    const uint4* ksrc = reinterpret_cast<const uint4*>(p.kc);
    uint4* kdst = reinterpret_cast<uint4*>(p.dkc);
    for (int i = tid; i < nt * p.bk; i += kMoveThreads) {
        const int t = i / p.bk, c = i - t * p.bk;
        if (s_dst[t] >= 0) kdst[s_dst[t] * p.bk + c] = ksrc[s_src[t] * p.bk + c];
    }
    // V records, a word a step: the even fields of one source, the odd ones of
    // the other (of a single last token: the record's own odd fields stay)
    const uint32_t* vsrc = reinterpret_cast<const uint32_t*>(p.vc);
    uint32_t* vdst = reinterpret_cast<uint32_t*>(p.dvc);
    constexpr int kW = 8 * BV;
    for (int i = tid; i < (nt + 1) / 2 * kW; i += kMoveThreads) {
        const int pr = i / kW, w = i - pr * kW;
        const int64_t dst = s_dst[2 * pr];
        if (dst < 0) continue;
        const uint32_t even = s_even[w];
        const int64_t sa = s_src[2 * pr];
        const uint32_t* ra = vsrc + (sa >> 1) * kW;
        uint32_t x = ra[w];
        if (sa & 1) x = __funnelshift_r(x, w + 1 < kW ? ra[w + 1] : 0u, BV);
        uint32_t* out = vdst + (dst >> 1) * kW + w;
        uint32_t y;
        if (2 * pr + 1 < nt) {
            const int64_t sb = s_src[2 * pr + 1];
            const uint32_t* rb = vsrc + (sb >> 1) * kW;
            y = rb[w];
            if (!(sb & 1)) y = __funnelshift_l(w > 0 ? rb[w - 1] : 0u, y, BV);
        } else {
            y = *out;
        }
        *out = (x & even) | (y & ~even);
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
        if (!done[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       kSelKeys * (int)sizeof(uint32_t));
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
    // a CTA for every kSelPerCta positions, up to a portable cluster
    int csize = 1;
    while (csize < kSelMaxCluster && (int64_t)csize * kSelPerCta < max_len) csize *= 2;
    const int64_t seg = ((max_len + csize - 1) / csize + 31) / 32 * 32;
    const int keys = seg <= kSelKeys ? (int)seg : 0;
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
    cfg.dynamicSmemBytes = (size_t)keys * sizeof(uint32_t);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, keys);
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
