// Appending keys and values to the 4-bit cache, the keys rotated on the way,
// and the cache's inspection.
//
// A group's image is put together in shared memory and stored as whole 16-byte
// pieces; of a group that is not new all through, the pieces that a new
// position touches are read first and the rest left alone, so no atomics and
// no other position's bytes change.  Heads run fastest over the blocks, so
// that the heads of a token find its cos and sin in L2.  Two kernels:
//   few groups   a block a group: eight threads a position for its keys, eight
//                for two positions' values (they share bytes), so that a thread
//                waits for its loads once (one token of 32 x 8 heads 3.4 us,
//                the other kernel 5.9)
//   many         a warp a group, its rows' loads all on their way at once
// Floor: 512 bytes in and 144 out for a token and head, 512 of tables a token.
// 131043 tokens of 2 heads, rotated: 51.5 us, 68 % of the copy bandwidth.  Bound by
// the bytes in flight: 128 registers leave 16 warps a SM, which spend 39 % of their
// time waiting for loads (issue slots 45 % busy).
#include <cuda_fp16.h>

#include "fp4.cuh"

namespace bgtq {
namespace {

constexpr int kKeyThreads = 8 * kGroup, kApThreads = kKeyThreads + 4 * kGroup;

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

__device__ __forceinline__ void load8(const __half* row, int d, uint32_t (&w)[4]) {
    const uint4 a = *reinterpret_cast<const uint4*>(row + d);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
}

// Codes of a piece of 8 key values (dims d .. d + 7 of position t) and, with the
// block's first half, its scale byte.
__device__ __forceinline__ void put_keys(uint8_t* img, int t, int d, const uint32_t (&x)[4], uint32_t byte, const Fp4Recip& r) {
    const uint32_t code = fp4_encode8(x, r);
    uint16_t* dst = reinterpret_cast<uint16_t*>(img + 64 * t + 32 * (d >> 3 & 1) + 2 * (d >> 4));
    dst[0] = (uint16_t)code;
    dst[8] = (uint16_t)(code >> 16);
    if (!(d & 8)) img[kGroupKs + 8 * t + (d >> 4)] = (uint8_t)byte;
}

// Block j of the values of positions t and t + 1 (t even; x: 16 values of each)
// of which those in `two` are new.
__device__ __forceinline__ void put_values(uint8_t* img, int t, int j, uint32_t two, const uint32_t (&x)[2][2][4]) {
    const int pc = (t >> 1) & 3, th = t >> 3;
    uint32_t code[2][2], s[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        s[e] = fp4_scale_byte(fmaxf(fp4_amax(x[e][0]), fp4_amax(x[e][1])));
        const Fp4Recip r(s[e]);
        code[e][0] = fp4_encode8(x[e][0], r);
        code[e][1] = fp4_encode8(x[e][1], r);
    }
    uint16_t* dst = reinterpret_cast<uint16_t*>(img + kGroupV + 512 * (j >> 2) + 16 * pc + 4 * (j & 3) + 2 * th);
    // byte of dim g of either half of the block: the two positions' codes
    constexpr uint32_t kEven = 0x0f0f0f0fu;
    uint32_t even[2], odd[2];  // dims 0 2 4 6 and 1 3 5 7 of both halves
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        even[hh] = (code[0][hh] & kEven) | ((code[1][hh] & kEven) << 4);
        odd[hh] = ((code[0][hh] >> 4) & kEven) | (code[1][hh] & ~kEven);
    }
    uint8_t* sd = img + kGroupVs + 32 * pc + 4 * j + 2 * th;
    if (two == 3u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t(&y)[2] = (i & 1) ? odd : even;
            dst[32 * i] = (uint16_t)__byte_perm(y[0], y[1], (i >> 1) | (4 + (i >> 1)) << 4 | 0x4400u);
        }
        *reinterpret_cast<uint16_t*>(sd) = (uint16_t)(s[0] | s[1] << 8);
    } else {
        const uint32_t keep = two == 1u ? 0xf0f0u : 0x0f0fu;  // nibbles of the other position
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t(&y)[2] = (i & 1) ? odd : even;
            const uint32_t u = __byte_perm(y[0], y[1], (i >> 1) | (4 + (i >> 1)) << 4 | 0x4400u);
            dst[32 * i] = (uint16_t)((u & ~keep) | (dst[32 * i] & keep));
        }
        if (two & 1u) sd[0] = (uint8_t)s[0];
        if (two & 2u) sd[1] = (uint8_t)s[1];
    }
}

__global__ void __launch_bounds__(kApThreads, 7) fp4_append_kernel(const __grid_constant__ Fp4AppendParams p) {
    __shared__ __align__(16) uint8_t img[kGroupBytes];
    __shared__ uint32_t s_fresh[kKeyThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31;
    const int h = (int)(blockIdx.x % (unsigned)p.map.H), b = blockIdx.y;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int ps = p.pos_start[b];
    if (ps < 0 || (int64_t)ps + p.t_new > p.cap) {
        if (blockIdx.x == 0 && tid == 0 && p.status) {
            atomicOr(p.status, BGTQ_STATUS_APPEND_CAPACITY);
            debug_in_range(false, p.status);  // positions past the capacity
        }
        return;
    }
    const int64_t end = (int64_t)ps + p.t_new;
    const int64_t gi = (ps >> 4) + (int64_t)(blockIdx.x / (unsigned)p.map.H);
    if (gi * kGroup >= end) return;
    const int row0 = (int)(gi * kGroup - ps);  // row of the group's first position (may be negative)
    uint8_t* g = p.map.group(b, h, gi);
    if (!g) {
        if (tid == 0 && p.status) atomicOr(p.status, BGTQ_STATUS_PAGE_RANGE);
        return;
    }
    // positions of the group that are given (bit i: position 16 gi + i)
    const int given_lo = max(0, -row0), given_hi = min(kGroup, p.t_new - row0);
    const uint32_t given = ((1u << given_hi) - 1u) & ~((1u << given_lo) - 1u);
    // ---- loads, pieces of 8 values.  Keys: thread i of a position has both dims of
    // blocks 8 i .. 8 i + 7; values: thread i has dims 16 i .. of two positions.
    const bool values = tid >= kKeyThreads;
    const bool halves = !p.rope.cos || p.rope.layout == 0;
    const int i8 = tid & 7, t = values ? 2 * ((tid - kKeyThreads) >> 3) : tid >> 3;
    const int da = values ? 16 * i8 : halves ? 8 * i8 : 16 * i8, db = values || !halves ? da + 8 : 64 + 8 * i8;
    uint32_t x[2][2][4] = {};
    int rp[2][kMaxAxes];
    uint32_t two = (given >> t) & (values ? 3u : 1u);  // which of the thread's positions are new
    {
        const RowsView& v = values ? p.v : p.k;
        const __half* base = static_cast<const __half*>(v.p) + b * v.sb + h * v.sh;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if ((two >> e) & 1u) {
                load8(base + (int64_t)(row0 + t + e) * v.st, da, x[e][0]);
                load8(base + (int64_t)(row0 + t + e) * v.st, db, x[e][1]);
            }
    }
    uint4 old = make_uint4(0u, 0u, 0u, 0u);
    const bool keeps = given != 0xffffu && tid < kGroupBytes / 16 && (given & piece_positions(tid));
    if (keeps) old = reinterpret_cast<const uint4*>(g)[tid];
    if (p.rope.cos) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (((two >> e) & 1u) && !rope_positions(p.rope, (int64_t)b * p.t_new + row0 + t + e, ps + (int64_t)row0 + t + e, rp[e])) {
                two &= ~(1u << e);
                if (h == 0 && !values && i8 == 0 && p.status) atomicOr(p.status, BGTQ_STATUS_ROPE_RANGE);
            }
        if (!values && (two & 1u)) rope_rotate8(p.rope, rp[0], 8 * i8, x[0][0], x[0][1]);
    }
    if (!values) {
        const uint32_t m = __ballot_sync(0xffffffffu, two & 1u);
        if (lane == 0) s_fresh[tid >> 5] = (m & 1u) | (m >> 7 & 2u) | (m >> 14 & 4u) | (m >> 21 & 8u);
    }
    if (keeps) reinterpret_cast<uint4*>(img)[tid] = old;
    __syncthreads();
    const uint32_t fresh = s_fresh[0] | s_fresh[1] << 4 | s_fresh[2] << 8 | s_fresh[3] << 12;
    if (given == 0xffffu && fresh != 0xffffu) {
        // (a whole group of which some position is skipped: what is kept, read now)
        if (tid < kGroupBytes / 16) reinterpret_cast<uint4*>(img)[tid] = reinterpret_cast<const uint4*>(g)[tid];
        __syncthreads();
    }
    // ---- codes into the image
    if (!values) {
        // a block's other half is the next lane's, or (neighbouring dims) this lane's own
        float ma = fp4_amax(x[0][0]), mb = fp4_amax(x[0][1]);
        if (halves) {
            ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, 1));
            mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
        } else {
            ma = mb = fmaxf(ma, mb);
        }
        if (two & 1u) {
            const uint32_t sa = fp4_scale_byte(ma), sb = halves ? fp4_scale_byte(mb) : sa;
            put_keys(img, t, da, x[0][0], sa, Fp4Recip(sa));
            put_keys(img, t, db, x[0][1], sb, Fp4Recip(sb));
        }
    } else if (two) {
        put_values(img, t, i8, two, x);
    }
    __syncthreads();
    if (tid < kGroupBytes / 16 && (fresh & piece_positions(tid)))
        reinterpret_cast<uint4*>(g)[tid] = reinterpret_cast<const uint4*>(img)[tid];
}

constexpr int kBulkWarps = kFp4AppendWarps;

template <bool kRope, bool kHalves>  // kHalves: both dims of a rotary block are 64 apart (layout 0), or there is none
__global__ void __launch_bounds__(32 * kBulkWarps) fp4_append_bulk_kernel(const __grid_constant__ Fp4AppendParams p) {
    __shared__ __align__(16) uint8_t s_img[kBulkWarps][kGroupBytes];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i8 = lane & 7;
    const int h = (int)(blockIdx.x % (unsigned)p.map.H), b = blockIdx.y;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int ps = p.pos_start[b];
    if (ps < 0 || (int64_t)ps + p.t_new > p.cap) {
        if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) {
            atomicOr(p.status, BGTQ_STATUS_APPEND_CAPACITY);
            debug_in_range(false, p.status);  // positions past the capacity
        }
        return;
    }
    const int64_t end = (int64_t)ps + p.t_new;
    const int64_t gi = (ps >> 4) + (int64_t)(blockIdx.x / (unsigned)p.map.H) * kBulkWarps + warp;
    if (gi * kGroup >= end) return;
    const int row0 = (int)(gi * kGroup - ps);  // row of the group's first position (may be negative)
    const int given_lo = max(0, -row0), given_hi = min(kGroup, p.t_new - row0);
    const uint32_t given = ((1u << given_hi) - 1u) & ~((1u << given_lo) - 1u);
    // ---- loads.  Keys: lanes 8 x .. 8 x + 7 have position 4 it + x, lane i both dims of
    // its blocks 8 i ..; values: lane (x, i) dims 16 i .. of positions 2 x + 8 it (+ 1)
    const int ka = kHalves ? 8 * i8 : 16 * i8, kb = kHalves ? 64 + 8 * i8 : 16 * i8 + 8;
    const __half* kp = static_cast<const __half*>(p.k.p) + b * p.k.sb + h * p.k.sh + (int64_t)row0 * p.k.st;
    const __half* vp = static_cast<const __half*>(p.v.p) + b * p.v.sb + h * p.v.sh + (int64_t)row0 * p.v.st;
    uint32_t kx[4][2][4], vx[2][2][2][4];
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int t = 4 * it + (lane >> 3);
#pragma unroll
        for (int e = 0; e < 4; ++e) kx[it][0][e] = kx[it][1][e] = 0u;
        if ((given >> t) & 1u) {
            load8(kp + t * p.k.st, ka, kx[it][0]);
            load8(kp + t * p.k.st, kb, kx[it][1]);
        }
    }
    // a position's row in the tables, by the lane of that number
    int rp[kMaxAxes] = {};
    bool mine = lane < kGroup && ((given >> lane) & 1u);
    if (kRope && mine && !rope_positions(p.rope, (int64_t)b * p.t_new + row0 + lane, (int64_t)ps + row0 + lane, rp)) {
        mine = false;
        rp[0] = rp[1] = rp[2] = rp[3] = 0;  // (loaded, not used)
        if (h == 0 && p.status) atomicOr(p.status, BGTQ_STATUS_ROPE_RANGE);
    }
    // cos and sin of a pass, one pass ahead
    auto tables = [&](RopeTurn& turn, int it) {
        const int t = 4 * it + (lane >> 3);
        int tp[kMaxAxes];
        tp[0] = tp[1] = tp[2] = tp[3] = __shfl_sync(0xffffffffu, rp[0], t);
        if (p.rope.axes > 1) {
#pragma unroll
            for (int e = 1; e < kMaxAxes; ++e) tp[e] = __shfl_sync(0xffffffffu, rp[e], t);
        }
        turn.load(p.rope, tp, 8 * i8);
    };
    RopeTurn turn;
    if constexpr (kRope) tables(turn, 0);
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int t = 2 * (lane >> 3) + 8 * it + n;
#pragma unroll
            for (int e = 0; e < 4; ++e) vx[it][n][0][e] = vx[it][n][1][e] = 0u;
            if ((given >> t) & 1u) {
                load8(vp + t * p.v.st, 16 * i8, vx[it][n][0]);
                load8(vp + t * p.v.st, 16 * i8 + 8, vx[it][n][1]);
            }
        }
    uint8_t* g = p.map.group(b, h, gi);
    if (!g) {
        if (lane == 0 && p.status) atomicOr(p.status, BGTQ_STATUS_PAGE_RANGE);
        return;
    }
    const uint32_t fresh = __ballot_sync(0xffffffffu, mine);
    uint8_t* img = s_img[warp];
    if (fresh != 0xffffu) {
        for (int i = lane; i < kGroupBytes / 16; i += 32)
            if (fresh & piece_positions(i)) reinterpret_cast<uint4*>(img)[i] = reinterpret_cast<const uint4*>(g)[i];
        __syncwarp();
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int t = 4 * it + (lane >> 3);
        const bool is_new = (fresh >> t) & 1u;
        if constexpr (kRope) {
            RopeTurn next;
            if (it < 3) tables(next, it + 1);
            rope_turn8(turn, kHalves, kx[it][0], kx[it][1]);
            turn = next;
        }
        // a block's other half is the next lane's, or (neighbouring dims) this lane's own
        float ma = fp4_amax(kx[it][0]), mb = fp4_amax(kx[it][1]);
        if constexpr (kHalves) {
            ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, 1));
            mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
        } else {
            ma = mb = fmaxf(ma, mb);
        }
        if (is_new) {
            const uint32_t sa = fp4_scale_byte(ma), sb = kHalves ? fp4_scale_byte(mb) : sa;
            put_keys(img, t, ka, kx[it][0], sa, Fp4Recip(sa));
            put_keys(img, t, kb, kx[it][1], sb, Fp4Recip(sb));
        }
    }
#pragma unroll
    for (int it = 0; it < 2; ++it) {
        const int t = 2 * (lane >> 3) + 8 * it;
        const uint32_t two = (fresh >> t) & 3u;
        if (two) put_values(img, t, i8, two, vx[it]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < (kGroupBytes / 16 + 31) / 32; ++i) {
        const int at = lane + 32 * i;
        if (at < kGroupBytes / 16 && (fresh & piece_positions(at)))
            reinterpret_cast<uint4*>(g)[at] = reinterpret_cast<const uint4*>(img)[at];
    }
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
    p.map = make_fp4_map(c, batch, status);
    p.t_new = t_new;
    p.cap = c.capacity;
    p.pos_start = pos_start;
    p.status = status;
    const int64_t groups = fp4_append_groups(t_new, c.capacity);
    // Up to 16 groups a SM (two waves of blocks): the block-a-group kernel's short chain of
    // waits; beyond, the work counts (131043 tokens x 2 heads: 64 us with a block
    // a group, whose six warps each pay for the set-up).
    const bool bulk = groups * c.n_heads * batch > 16 * 152;
    const int64_t blocks = bulk ? fp4_append_blocks(groups, c.n_heads) : groups * c.n_heads;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)batch, 1);
    cfg.blockDim = dim3(bulk ? 32 * kBulkWarps : kApThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (!bulk) return cudaLaunchKernelEx(&cfg, fp4_append_kernel, p);
    if (!r.cos) return cudaLaunchKernelEx(&cfg, fp4_append_bulk_kernel<false, true>, p);
    return r.layout == 0 ? cudaLaunchKernelEx(&cfg, fp4_append_bulk_kernel<true, true>, p)
                         : cudaLaunchKernelEx(&cfg, fp4_append_bulk_kernel<true, false>, p);
}

cudaError_t launch_fp4_dequant(cudaStream_t s, const bgtq_fp4_cache& c, int batch, int b, int head, int64_t t0, int64_t t1, float* k_out,
                               float* v_out) {
    fp4_dequant_kernel<<<(unsigned)(t1 - t0), kD, 0, s>>>(make_fp4_map(c, batch, nullptr), b, head, t0, t1, k_out, v_out);
    return cudaGetLastError();
}

}  // namespace bgtq
