// The 4-bit cache: its groups, and the arithmetic of its codes and scales.
//
// Blocks of 16 values: 4-bit codes (e2m1) under an 8-bit scale whose byte is
// bits 14..7 of an fp16 number (5 exponent bits, 3 mantissa bits), so that a
// scale becomes fp16 by a shift, a code by the hardware's conversion, and
// their product (2 + 4 significant bits, never below 2^-18) is exact in fp16:
// no second scale for the row, no rounding when the cache is read.  A group
// holds 16 positions of one head, keys and values, in the order in which the
// lanes of an m16n8k16 product want them (bgtq.h gives the byte of every
// value): 2304 contiguous bytes, which one bulk copy brings in.
#pragma once

#include "rope.cuh"

namespace bgtq {

constexpr int kGroup = 16;           // positions of a group
constexpr int kGroupBytes = 2304;
constexpr int kGroupV = 1024;        // value codes
constexpr int kGroupKs = 2048;       // key scales
constexpr int kGroupVs = 2176;       // value scales
constexpr int kScaleMax = 226;       // byte of 10240: 6 x 10240 is finite in fp16

struct Fp4Map {
    uint8_t* base;
    const int32_t* page_table;  // [B][max_pages], nullptr: contiguous
    int64_t cap_groups;         // groups of a sequence
    int64_t max_pages, n_pages;
    int H, lg;                  // lg = log2(P / 16)
    int batch;                  // sequences of the launch
    int32_t* status;            // where a failed range check is reported
#ifdef __CUDACC__
    // nullptr when the page_table entry is outside [0, n_pages) (and, in the
    // BGTQ_DEBUG_BOUNDS build, when b, h or gi is out of range)
    __device__ __forceinline__ uint8_t* group(int b, int h, int64_t gi) const {
        if (!debug_in_range(b >= 0 && b < batch && h >= 0 && h < H && gi >= 0 && gi < cap_groups, status)) return nullptr;
        if (!page_table) return base + (((int64_t)b * H + h) * cap_groups + gi) * kGroupBytes;
        const int32_t pg = page_table[(int64_t)b * max_pages + (gi >> lg)];
        if (pg < 0 || (int64_t)pg >= n_pages) {
            debug_in_range(false, status);
            return nullptr;
        }
        return base + ((((int64_t)pg * H + h) << lg) + (gi & (((int64_t)1 << lg) - 1))) * kGroupBytes;
    }
#endif
};

inline Fp4Map make_fp4_map(const bgtq_fp4_cache& c, int batch, int32_t* status) {
    Fp4Map m;
    m.base = static_cast<uint8_t*>(c.groups);
    m.page_table = c.page_table;
    m.cap_groups = c.capacity / kGroup;
    m.max_pages = c.page_table ? c.max_pages : 1;
    m.n_pages = c.page_table ? c.n_pages : 1;
    m.H = c.n_heads;
    m.lg = 0;
    if (c.page_table)
        while (((int64_t)kGroup << m.lg) < c.page_tokens) ++m.lg;
    m.batch = batch;
    m.status = status;
    return m;
}

// What bgtq_fp4_attn runs: the one-pass kernel (fp4_attn.cu) for up to
// kFp4RowsLeast query rows of a KV head and, where there is work enough, up to
// kFp4Rows; else the tensor cores' tiles (fp4_tiles.cu).
constexpr int kFp4RowsLeast = 16, kFp4Rows = 32;
struct Fp4Attn {
    RopeParams rope;
    RowsView q;
    Fp4Map map;
    const int32_t* seq_lens;
    int64_t cap, max_len;
    int batch, t, group;
    void* out;
    int out_dtype;
    float scale;
    void* ws;
    int32_t* status;
};
size_t fp4_attn_workspace_bytes(int H, int group, int batch, int t, int64_t max_len);
cudaError_t launch_fp4_attn(cudaStream_t s, const Fp4Attn& a);
// The tiles' part (fp4_tiles.cu); ws behind the counters of the one-pass kernel.
size_t fp4_tiles_workspace_bytes(int64_t heads, int64_t rows, int64_t max_len);
cudaError_t launch_fp4_tiles(cudaStream_t s, const Fp4Attn& a, void* ws);
// Groups of a sequence that t_new positions can touch (more than the capacity:
// no sequence takes them, and the kernels' first blocks say so), and the blocks
// of the warp-a-group append of all heads.
constexpr int kFp4AppendWarps = 4;
inline int64_t fp4_append_groups(int64_t t_new, int64_t capacity) { return ((t_new < capacity ? t_new : capacity) + kGroup - 2) / kGroup + 1; }
inline int64_t fp4_append_blocks(int64_t groups, int heads) { return (groups + kFp4AppendWarps - 1) / kFp4AppendWarps * heads; }
cudaError_t launch_fp4_append(cudaStream_t s, const RopeParams& r, const RowsView& k, const RowsView& v, int batch, int t_new,
                              const int32_t* pos_start, const bgtq_fp4_cache& c, int32_t* status);
cudaError_t launch_fp4_dequant(cudaStream_t s, const bgtq_fp4_cache& c, int batch, int b, int head, int64_t t0, int64_t t1, float* k_out,
                               float* v_out);

#ifdef __CUDACC__
namespace {

// Two neighbouring scale bytes (of `w`, at bytes lo and lo + 1) as two fp16.
template <int kLo>
__device__ __forceinline__ __half2 fp4_scales(uint32_t w) {
    const uint32_t u = __byte_perm(w, 0u, kLo == 0 ? 0x4140 : 0x4342) << 7;
    return *reinterpret_cast<const __half2*>(&u);
}

// The four code pairs of a word: byte i gives the numbers of its low and high nibble.
__device__ __forceinline__ void fp4_numbers(uint32_t w, __half2 (&x)[4]) {
    uint32_t u[4];
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const __half2*>(&u[i]);
}

// Byte of the scale of a block whose largest magnitude is amax: amax / 6 to
// four significant bits, ties to even, steps of 2^-17 below 2^-14.  The
// quotient comes from 1/6 in two parts, the first of 12 bits, whose product
// with amax (11 bits) is exact: a quotient that is a tie (five bits) comes out
// as that tie, and any other is at least 2^-12 of itself away from one.
__device__ __forceinline__ uint32_t fp4_scale_byte(float amax) {
    constexpr float kHi = 0.1666259765625f, kLo = (float)(1.0 / 6.0 - 0.1666259765625);
    const float y = __fmaf_rn(amax, kLo, __fmul_rn(amax, kHi));
    const uint32_t u = __float_as_uint(y);
    const uint32_t norm = ((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - (112u << 3);
    const uint32_t sub = (uint32_t)__float2int_rn(__fmul_rn(y, 131072.0f));
    return min(y < 6.103515625e-5f ? sub : norm, (uint32_t)kScaleMax);
}

__device__ __forceinline__ float fp4_amax(const uint32_t (&w)[4]) {
    const __half2 m = __hmax2(__hmax2(__habs2(*reinterpret_cast<const __half2*>(&w[0])), __habs2(*reinterpret_cast<const __half2*>(&w[1]))),
                              __hmax2(__habs2(*reinterpret_cast<const __half2*>(&w[2])), __habs2(*reinterpret_cast<const __half2*>(&w[3]))));
    return fmaxf(__low2float(m), __high2float(m));
}

// A block's reciprocal scale in two parts, the first of 12 bits (0 for scale 0).
struct Fp4Recip {
    uint64_t hi, lo;  // each twice
    __device__ __forceinline__ explicit Fp4Recip(uint32_t byte) {
        const float s = __half2float(__ushort_as_half((unsigned short)(byte << 7)));
        const float r = byte ? __frcp_rn(s) : 0.0f;
        const float h = __uint_as_float(__float_as_uint(r) & 0xfffff000u);
        const float l = byte ? __fmul_rn(__fmaf_rn(-h, s, 1.0f), r) : 0.0f;
        hi = pair2(h, h);
        lo = pair2(l, l);
    }
};

// Half a block, 8 fp16 values (4 words) -> 8 codes in dim order.  x/s = x hi +
// x lo: the first product is exact (11 and 12 bits), so the sum is the quotient
// to 2^-36 rounded once to fp32.  A quotient that is a midpoint of two codes
// comes out as that midpoint, and any other is at least 2^-18 of itself away
// from one (x has 11 bits, s four, a midpoint three).  A zero keeps its sign.
__device__ __forceinline__ uint32_t fp4_encode8(const uint32_t (&w)[4], const Fp4Recip& r) {
    float2 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = rope_f2(w[i]);
        const uint64_t p = pair2(x.x, x.y);
        q[i] = halves2(fma_pair(p, r.lo, mul_pair(p, r.hi)));
    }
    uint32_t c;
    asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
        : "=r"(c)
        : "f"(q[0].x), "f"(q[0].y), "f"(q[1].x), "f"(q[1].y), "f"(q[2].x), "f"(q[2].y), "f"(q[3].x), "f"(q[3].y));
    return c;
}

}  // namespace
#endif

}  // namespace bgtq
