// Decode attention that adds its weights to a score per cached position: the
// scoring instances of the decode kernel on a contiguous packed cache
// (decode_kernel.cuh) and the score kernel.
//
// score_j += sum_g p_gj, p_gj = 2^(l_gj - m_g) / L_g: a weight needs the
// softmax statistics of the whole row, which no split knows before the merge.
// The decode launch therefore writes every logit (fp32, 4 G bytes per cached
// token and KV head, against 16 bK + 16 bV + 8 of packed records) and the
// merged (m, L); a second launch turns them into weights.  At a cache of 128K
// tokens the logits of a layer are 8 MB and stay in the 129 MB L2 between the
// two launches.  Sums run over the query heads in order: no atomics.
#include <algorithm>

#include "decode_kernel.cuh"

namespace bgtq {
namespace {

struct ScoreParams {
    const float* logit;  // [B][H][G][stride], log2 domain
    int64_t stride;
    const float2* stat;  // [B][H][G] (maximum, sum)
    const int32_t* seq_lens;
    const int32_t* pos_new;  // nullptr: attention only
    const float* in;
    float* out;
    int64_t cap;  // row length of in and out
    int64_t max_seq;
    int H, G;
};

constexpr int kScoreThreads = 256;
constexpr int kScoreTok = 2;  // positions per thread (8-byte accesses: rows start 8-byte aligned)

__global__ void __launch_bounds__(kScoreThreads) score_add_kernel(ScoreParams p) {
    pdl_trigger();
    const int h = blockIdx.y, b = blockIdx.z;
    const size_t unit = (size_t)b * p.H + h;
    const int seq = (int)min((int64_t)max(p.seq_lens[b], 0), p.max_seq);  // as the decode launch cuts it
    const int t0 = (blockIdx.x * kScoreThreads + threadIdx.x) * kScoreTok;
    const int fresh = p.pos_new ? p.pos_new[b] : -1;  // a new position has no weight yet
    pdl_wait();  // the logits, and the scores a previous kernel may be writing
    // a new position that this step does not attend (at or past the length)
    // starts at 0 as well: no other call would set it
    if (fresh >= seq && fresh < p.cap && blockIdx.x == 0 && threadIdx.x == 0) p.out[unit * (size_t)p.cap + fresh] = 0.0f;
    if (t0 >= seq) return;
    // every head's statistics and logits in flight at once, then the sums in
    // the heads' order
    const float* lg = p.logit + unit * p.G * (size_t)p.stride + t0;
    float2 st[8], l[8];
#pragma unroll
    for (int g = 0; g < 8; ++g) {
        if (g >= p.G) break;
        st[g] = p.stat[unit * p.G + g];
        l[g] = __ldcs(reinterpret_cast<const float2*>(lg + g * (size_t)p.stride));
    }
    float w0 = 0.0f, w1 = 0.0f;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
        if (g >= p.G) break;
        const float inv = 1.0f / st[g].y;
        w0 += fast_exp2(l[g].x - st[g].x) * inv;
        w1 += fast_exp2(l[g].y - st[g].x) * inv;
    }
    const size_t at = unit * (size_t)p.cap + t0;
    if (t0 + 1 < seq) {
        const float2 was = *reinterpret_cast<const float2*>(p.in + at);
        *reinterpret_cast<float2*>(p.out + at) =
            make_float2((t0 == fresh ? 0.0f : was.x) + w0, (t0 + 1 == fresh ? 0.0f : was.y) + w1);
    } else {
        p.out[at] = (t0 == fresh ? 0.0f : p.in[at]) + w0;
    }
}

}  // namespace

cudaError_t launch_decode_score(const DecodeParams& p, dim3 grid, cudaStream_t s, int kind, int bk, int bv) {
    return launch_widths<false, kDecodeScore>(p, grid, s, kind, bk, bv);
}

cudaError_t launch_score_add(const bgtq_plan& pl, cudaStream_t s, const bgtq_cache& c, const int32_t* seq_lens,
                             int64_t max_len, int batch, const DecodeExtra& extra, const int32_t* pos_new,
                             const float* scores_in, float* scores_out) {
    if (max_len == 0 && !pos_new) return cudaSuccess;
    ScoreParams p;
    p.logit = extra.logit;
    p.stride = extra.logit_stride;
    p.stat = extra.stat;
    p.seq_lens = seq_lens;
    p.pos_new = pos_new;
    p.in = scores_in;
    p.out = scores_out;
    p.cap = c.capacity;
    p.max_seq = max_len;
    p.H = pl.H;
    p.G = pl.G;
    constexpr int64_t per_block = kScoreThreads * kScoreTok;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::max<int64_t>(1, (max_len + per_block - 1) / per_block), (unsigned)pl.H, (unsigned)batch);
    cfg.blockDim = dim3(kScoreThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, score_add_kernel, p);
}

}  // namespace bgtq
