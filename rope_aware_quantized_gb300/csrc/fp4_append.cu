// Appending keys and values to the 4-bit cache, the keys rotated on the way,
// and the cache's inspection.
//
// One warp writes one group: 16 positions of a head, keys and values.  Its
// image is put together in shared memory and stored as whole 16-byte pieces;
// of a group that is not new all through, the pieces that a new position
// touches are read first and the rest left alone, so no atomics and no other
// position's bytes change.  Heads run fastest over the blocks, so that the
// heads of a token find its cos and sin in L2.
// Bound by HBM: 512 bytes in and 144 out for a token and head (and 512 of
// tables a token), about 60 warp-instructions.
#include <cuda_fp16.h>

#include "fp4.cuh"

namespace bgtq {
namespace {

constexpr int kApWarps = 4;

struct Fp4AppendParams {
    RopeParams rope;
    RowsView k, v;
    Fp4Map map;
    int t_new;
    int64_t cap;
    const int32_t* pos_start;
    int32_t* status;
};

// Positions of a group (bits of the mask) whose bytes lie in its 16-byte piece i.
__device__ __forceinline__ uint32_t piece_positions(int i) {
    if (i < 64) return 1u << (i >> 2);
    if (i < 128) return 0x303u << (2 * (i & 3));
    if (i < 136) return 3u << (2 * (i - 128));
    return 0x303u << (2 * ((i - 136) >> 1));
}

__device__ __forceinline__ void load16(const __half* row, int d, uint32_t (&w)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(row + d), b = *reinterpret_cast<const uint4*>(row + d + 8);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}

__global__ void __launch_bounds__(32 * kApWarps) fp4_append_kernel(const __grid_constant__ Fp4AppendParams p) {
    __shared__ __align__(16) uint8_t s_img[kApWarps][kGroupBytes];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = (int)(blockIdx.x % (unsigned)p.map.H), b = blockIdx.y;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int ps = p.pos_start[b];
    if (ps < 0 || (int64_t)ps + p.t_new > p.cap) {
        if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) atomicOr(p.status, BGTQ_STATUS_APPEND_CAPACITY);
        return;
    }
    const int64_t end = (int64_t)ps + p.t_new;
    const int64_t gi = (ps >> 4) + (int64_t)(blockIdx.x / (unsigned)p.map.H) * kApWarps + warp;
    if (gi * kGroup >= end) return;
    // which of the group's positions are new (bit i: position 16 gi + i)
    int rp[kMaxAxes] = {};
    bool mine = false;
    if (lane < kGroup) {
        const int64_t pos = gi * kGroup + lane;
        mine = pos >= ps && pos < end;
        if (mine && p.rope.cos && !rope_positions(p.rope, (int64_t)b * p.t_new + (pos - ps), pos, rp)) {
            mine = false;
            if (h == 0 && p.status) atomicOr(p.status, BGTQ_STATUS_ROPE_RANGE);
        }
    }
    const uint32_t fresh = __ballot_sync(0xffffffffu, mine);
    if (fresh == 0) return;
    uint8_t* g = p.map.group(b, h, gi);
    if (!g) {
        if (lane == 0 && p.status) atomicOr(p.status, BGTQ_STATUS_PAGE_RANGE);
        return;
    }
    uint8_t* img = s_img[warp];
    if (fresh != 0xffffu) {
        for (int i = lane; i < kGroupBytes / 16; i += 32)
            if (fresh & piece_positions(i)) reinterpret_cast<uint4*>(img)[i] = reinterpret_cast<const uint4*>(g)[i];
        __syncwarp();
    }
    const int64_t row0 = gi * kGroup - ps;  // row of the group's first position
    // ---- keys: a lane takes blocks j and j + 4 of a token (both dims of a
    // rotary block in either layout)
    const __half* kb = static_cast<const __half*>(p.k.p) + b * p.k.sb + h * p.k.sh;
#pragma unroll
    for (int it = 0; it < 2; ++it) {
        const int t = 8 * it + (lane >> 2), j = lane & 3;
        int tp[kMaxAxes];
        if (p.rope.cos) {
#pragma unroll
            for (int a = 0; a < kMaxAxes; ++a) tp[a] = __shfl_sync(0xffffffffu, rp[a], t);
        }
        if (!((fresh >> t) & 1u)) continue;
        const __half* row = kb + (row0 + t) * p.k.st;
        uint32_t a[8], c[8];
        load16(row, 16 * j, a);
        load16(row, 64 + 16 * j, c);
        if (p.rope.cos) {
            uint32_t(&a0)[4] = *reinterpret_cast<uint32_t(*)[4]>(&a[0]);
            uint32_t(&a1)[4] = *reinterpret_cast<uint32_t(*)[4]>(&a[4]);
            uint32_t(&c0)[4] = *reinterpret_cast<uint32_t(*)[4]>(&c[0]);
            uint32_t(&c1)[4] = *reinterpret_cast<uint32_t(*)[4]>(&c[4]);
            if (p.rope.layout == 0) {
                rope_rotate8(p.rope, tp, 16 * j, a0, c0);
                rope_rotate8(p.rope, tp, 16 * j + 8, a1, c1);
            } else {
                rope_rotate8(p.rope, tp, 8 * j, a0, a1);
                rope_rotate8(p.rope, tp, 32 + 8 * j, c0, c1);
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t code[2];
            const uint32_t s = fp4_encode(half ? c : a, code);
            uint16_t* dst = reinterpret_cast<uint16_t*>(img + 64 * t + 2 * (j + 4 * half));
            dst[0] = (uint16_t)code[0];
            dst[8] = (uint16_t)(code[0] >> 16);
            dst[16] = (uint16_t)code[1];
            dst[24] = (uint16_t)(code[1] >> 16);
            img[kGroupKs + 8 * t + j + 4 * half] = (uint8_t)s;
        }
    }
    // ---- values: a lane takes block j of two neighbouring tokens, which share bytes
    const __half* vb = static_cast<const __half*>(p.v.p) + b * p.v.sb + h * p.v.sh;
#pragma unroll
    for (int it = 0; it < 2; ++it) {
        const int pc = lane >> 3, j = lane & 7, t = 2 * pc + 8 * it;
        const uint32_t two = (fresh >> t) & 3u;
        if (two == 0) continue;
        uint32_t code[2][2] = {}, s[2] = {};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            if (!((two >> n) & 1u)) continue;
            uint32_t w[8];
            load16(vb + (row0 + t + n) * p.v.st, 16 * j, w);
            s[n] = fp4_encode(w, code[n]);
        }
        uint16_t* dst = reinterpret_cast<uint16_t*>(img + kGroupV + 512 * (j >> 2) + 16 * pc + 4 * (j & 3) + 2 * it);
        const uint32_t keep = two == 3u ? 0u : two == 1u ? 0xf0f0u : 0x0f0fu;  // nibbles of the other token
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t u = ((code[0][0] >> (4 * i)) & 15u) | ((code[1][0] >> (4 * i)) & 15u) << 4 |
                         ((code[0][1] >> (4 * i)) & 15u) << 8 | ((code[1][1] >> (4 * i)) & 15u) << 12;
            if (keep) u |= dst[32 * i] & keep;
            dst[32 * i] = (uint16_t)u;
        }
        uint8_t* sd = img + kGroupVs + 32 * pc + 4 * j + 2 * it;
        if (two & 1u) sd[0] = (uint8_t)s[0];
        if (two & 2u) sd[1] = (uint8_t)s[1];
    }
    __syncwarp();
    for (int i = lane; i < kGroupBytes / 16; i += 32)
        if (fresh & piece_positions(i)) reinterpret_cast<uint4*>(g)[i] = reinterpret_cast<const uint4*>(img)[i];
}

// One thread a dim of a position.
__global__ void __launch_bounds__(128) fp4_dequant_kernel(Fp4Map map, int b, int h, int64_t t0, int64_t t1, float* ko, float* vo) {
    const int64_t pos = t0 + blockIdx.x;
    const int d = threadIdx.x, t = (int)(pos & 15);
    const uint8_t* g = map.group(b, h, pos >> 4);
    const int64_t at = (pos - t0) * kD + d;
    auto value = [](uint32_t nibble, uint32_t scale) {
        __half2 x[4];
        fp4_numbers(nibble, x);
        return __half2float(__hmul(__low2half(x[0]), __ushort_as_half((unsigned short)(scale << 7))));
    };
    if (ko) {
        float x = 0.0f;
        if (g) x = value((g[64 * t + 16 * (d / 4 % 4) + 2 * (d / 16) + d / 2 % 2] >> (4 * (d & 1))) & 15u, g[kGroupKs + 8 * t + d / 16]);
        ko[at] = x;
    }
    if (vo) {
        float x = 0.0f;
        if (g)
            x = value((g[kGroupV + 512 * (d / 64) + 64 * (d % 8) + 16 * (t / 2 % 4) + 4 * (d / 16 % 4) + 2 * (t / 8) + d / 8 % 2] >>
                       (4 * (t & 1))) & 15u,
                      g[kGroupVs + 32 * (t / 2 % 4) + 4 * (d / 16) + 2 * (t / 8) + (t & 1)]);
        vo[at] = x;
    }
}

}  // namespace

cudaError_t launch_fp4_append(cudaStream_t s, const RopeParams& r, const RowsView& k, const RowsView& v, int batch, int t_new,
                              const int32_t* pos_start, const bgtq_fp4_cache& c, int32_t* status) {
    Fp4AppendParams p;
    p.rope = r;
    p.k = k;
    p.v = v;
    p.map = make_fp4_map(c);
    p.t_new = t_new;
    p.cap = c.capacity;
    p.pos_start = pos_start;
    p.status = status;
    const int64_t groups = ((int64_t)t_new + 14) / kGroup + 1;  // that t_new positions can touch
    const int64_t blocks = (groups + kApWarps - 1) / kApWarps * c.n_heads;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)batch, 1);
    cfg.blockDim = dim3(32 * kApWarps, 1, 1);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fp4_append_kernel, p);
}

cudaError_t launch_fp4_dequant(cudaStream_t s, const bgtq_fp4_cache& c, int b, int head, int64_t t0, int64_t t1, float* k_out,
                               float* v_out) {
    fp4_dequant_kernel<<<(unsigned)(t1 - t0), kD, 0, s>>>(make_fp4_map(c), b, head, t0, t1, k_out, v_out);
    return cudaGetLastError();
}

}  // namespace bgtq
