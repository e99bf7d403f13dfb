// Rotary positions: the tables' view on the device and the rotation of one
// 2-D block, shared by every kernel that rotates rows.
//
// "Under RoPE a key's contribution to a logit is a sum over 2-D frequency
// blocks" (English abstract): block i of 64 is the dims (i, i + 64) or
// (2i, 2i + 1), turned by the angle of the row's position on the block's axis.
// Every operation is one correctly rounded float32 operation, so a row's
// rotated bits do not depend on the kernel that rotates it.
#pragma once

#include <cuda_fp16.h>
#include <limits.h>

#include "bgtq_internal.h"

namespace bgtq {

constexpr int kMaxAxes = 4;

struct RopeParams {
    const float* cos;    // [n_pos][64]; nullptr: rows are taken as they are
    const float* sin;
    const int32_t* pos;  // [axes][batch * t]; nullptr: the row's own position on every axis
    int64_t pos_rows;    // batch * t
    int n_pos;
    int axes;
    int layout;
    uint32_t axis2[4];   // axis of block i: bits 2 (i mod 16) of word i / 16
};

// Strided rows (b, h, i) of 128 elements
struct RowsView {
    const void* p;
    int64_t sb, sh, st;
};

// Kernel view of a host descriptor (rope NULL: no rotation).
inline RopeParams make_rope(const bgtq_rope* r, const int32_t* pos, int64_t rows) {
    RopeParams p = {};
    if (!r) return p;
    p.cos = r->cos;
    p.sin = r->sin;
    p.pos = pos;
    p.pos_rows = rows;
    p.n_pos = (int)r->n_pos;
    p.axes = r->axes;
    p.layout = r->layout;
    for (int i = 0; i < kNB; ++i)
        if (r->axis) p.axis2[i >> 4] |= (uint32_t)(r->axis[i] & 3) << (2 * (i & 15));
    return p;
}
inline RowsView make_rows(const bgtq_rows& r) { return {r.data, r.stride_b, r.stride_h, r.stride_t}; }

// Host checks (rope_host.cpp); they set the thread's error message.
int check_rope(const bgtq_rope* r);
// Rows of `elem`-byte elements: pointer and strides 16-byte aligned; of an
// output also that no two rows meet.
int check_rows(const bgtq_rows* r, const char* name, int batch, int heads, int64_t t, int elem, bool output);

#ifdef __CUDACC__
namespace {

// Two floats as one operand: each operation rounds both as its scalar does.
__device__ __forceinline__ uint64_t pair2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 halves2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// The row's position on each axis; false when one lies outside the tables.
__device__ __forceinline__ bool rope_positions(const RopeParams& r, int64_t row, int64_t own, int (&pos)[kMaxAxes]) {
    if (!r.pos || r.axes == 1) {
        // (one axis, or the row's own position on all of them)
        const int v = r.pos ? r.pos[row] : own < INT_MAX ? (int)own : -1;
#pragma unroll
        for (int a = 0; a < kMaxAxes; ++a) pos[a] = v;
        return (uint32_t)v < (uint32_t)r.n_pos;
    }
    bool ok = true;
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a) {
        const int v = r.pos[a < r.axes ? a * r.pos_rows + row : row];
        ok = ok && (uint32_t)v < (uint32_t)r.n_pos;
        pos[a] = v;
    }
    return ok;
}

__device__ __forceinline__ int rope_pick(const int (&pos)[kMaxAxes], uint32_t a) {
    return a < 2 ? (a ? pos[1] : pos[0]) : (a == 2 ? pos[2] : pos[3]);
}

// cos and sin of blocks i0 .. i0 + 3 (i0 a multiple of 4) at the row's
// positions: one 16-byte load each when the four lie on one axis.
__device__ __forceinline__ void rope_load4(const RopeParams& r, const int (&pos)[kMaxAxes], int i0, float (&c)[4], float (&s)[4]) {
    const uint32_t ax = r.axes == 1 ? 0u : (r.axis2[i0 >> 4] >> (2 * (i0 & 15))) & 0xffu;
    if (ax == (ax & 3u) * 0x55u) {
        const int64_t at = (int64_t)rope_pick(pos, ax & 3u) * kNB + i0;
        const float4 cv = __ldg(reinterpret_cast<const float4*>(r.cos + at));
        const float4 sv = __ldg(reinterpret_cast<const float4*>(r.sin + at));
        c[0] = cv.x, c[1] = cv.y, c[2] = cv.z, c[3] = cv.w;
        s[0] = sv.x, s[1] = sv.y, s[2] = sv.z, s[3] = sv.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t at = (int64_t)rope_pick(pos, (ax >> (2 * k)) & 3u) * kNB + i0 + k;
            c[k] = __ldg(r.cos + at);
            s[k] = __ldg(r.sin + at);
        }
    }
}

__device__ __forceinline__ void rope_pair(float& lo, float& hi, float c, float s) {
    const float a = __fsub_rn(__fmul_rn(lo, c), __fmul_rn(hi, s));
    hi = __fadd_rn(__fmul_rn(hi, c), __fmul_rn(lo, s));
    lo = a;
}

// One element of a rotated fp16 row: dim d of row x.
__device__ __forceinline__ __half rope_elem(const RopeParams& r, const int (&pos)[kMaxAxes], const __half* x, int d) {
    const int i = r.layout ? d >> 1 : d & 63;
    const int dl = r.layout ? 2 * i : i, dh = r.layout ? 2 * i + 1 : i + 64;
    const uint32_t ax = (r.axis2[i >> 4] >> (2 * (i & 15))) & 3u;
    const int64_t at = (int64_t)rope_pick(pos, ax) * kNB + i;
    float lo = __half2float(x[dl]), hi = __half2float(x[dh]);
    rope_pair(lo, hi, __ldg(r.cos + at), __ldg(r.sin + at));
    return __float2half_rn(d == dl ? lo : hi);
}

__device__ __forceinline__ uint32_t rope_h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 rope_f2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// cos and sin of blocks i0 .. i0 + 7.
struct RopeTurn {
    float c[8], s[8];
    __device__ __forceinline__ void load(const RopeParams& r, const int (&pos)[kMaxAxes], int i0) {
        rope_load4(r, pos, i0, *reinterpret_cast<float(*)[4]>(&c[0]), *reinterpret_cast<float(*)[4]>(&s[0]));
        rope_load4(r, pos, i0 + 4, *reinterpret_cast<float(*)[4]>(&c[4]), *reinterpret_cast<float(*)[4]>(&s[4]));
    }
};

// Turn blocks i0 .. i0 + 7 of an fp16 row held as 8 words: halves, a = dims i0
// .. i0 + 7 and b = dims 64 + i0 .. (layout 0); else a and b = dims 2 i0 .. 2 i0 + 15.
__device__ __forceinline__ void rope_turn8(const RopeTurn& t, bool halves, uint32_t (&a)[4], uint32_t (&b)[4]) {
    if (halves) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float2 x = rope_f2(a[m]), y = rope_f2(b[m]);
            const uint64_t lo = pair2(x.x, x.y), hi = pair2(y.x, y.y);
            const uint64_t cc = pair2(t.c[2 * m], t.c[2 * m + 1]), ss = pair2(t.s[2 * m], t.s[2 * m + 1]);
            // (the sums one by one: a packed product and a packed sum came out as one
            // rounding where the compiler may contract them)
            const float2 lc = halves2(mul_pair(lo, cc)), hs = halves2(mul_pair(hi, ss));
            const float2 hc = halves2(mul_pair(hi, cc)), ls = halves2(mul_pair(lo, ss));
            a[m] = rope_h2(__fsub_rn(lc.x, hs.x), __fsub_rn(lc.y, hs.y));
            b[m] = rope_h2(__fadd_rn(hc.x, ls.x), __fadd_rn(hc.y, ls.y));
        }
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t(&w)[4] = k ? b : a;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                float2 x = rope_f2(w[m]);
                rope_pair(x.x, x.y, t.c[4 * k + m], t.s[4 * k + m]);
                w[m] = rope_h2(x.x, x.y);
            }
        }
    }
}

__device__ __forceinline__ void rope_rotate8(const RopeParams& r, const int (&pos)[kMaxAxes], int i0, uint32_t (&a)[4], uint32_t (&b)[4]) {
    RopeTurn t;
    t.load(r, pos, i0);
    rope_turn8(t, r.layout == 0, a, b);
}

}  // namespace
#endif

// Launchers (they only enqueue work).
cudaError_t launch_rope_table(cudaStream_t s, const double* inv_freq, int64_t n_pos, double scale, float* cos, float* sin);
// Rows of q and k, each (input, output, heads).
cudaError_t launch_rope_rows(cudaStream_t s, const RopeParams& r, int batch, int t, const RowsView& q, const RowsView& q_out,
                             int n_q, const RowsView& k, const RowsView& k_out, int n_k, int in_dtype, int out_dtype,
                             int inverse, int32_t* status);
cudaError_t launch_rope_append(const bgtq_plan& p, cudaStream_t s, const RopeParams& r, const RowsView& k, const RowsView& v,
                               int batch, int t_new, const int32_t* pos_start, const bgtq_cache& c, int32_t* status);

}  // namespace bgtq
