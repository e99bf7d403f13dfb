// Rotary tables and the rotation of queries and keys.
//
// RoPE turns every 2-D frequency block of a query or key by an angle of its
// position ("RoPE-Aware Bit Allocation for KV-Cache Quantization", English
// abstract: a logit is a sum over those blocks).  On several axes (time,
// height, width) each block takes the position of its own axis.
//
// rope_rows: bound by HBM (each row read and written once, 3 flops an
// element).  A thread takes 8 blocks of one token (16 elements of a row), reads
// their cos and sin once and turns them in a share of the token's heads, two
// rows in flight; few tokens are shared out over more threads, head by head.
// 32768 tokens x 18 heads: 49.6 us, 0.95 of measured HBM (four rows in flight:
// 52.8, their registers halve the warps; 256 threads: 55.6).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rope.cuh"

namespace bgtq {
namespace {

struct FreqTable {
    double f[kNB];
};

// Angles and functions in float64: a float32 product of a far position and a
// frequency is off by whole radians' fractions (2^-24 of 10^6 rad).  Bound by the
// 64-bit functions: 131072 positions take 478 us (their bytes 10), 4096 16 us; a
// model's tables are made once.
__global__ void __launch_bounds__(256) rope_table_kernel(FreqTable f, int64_t n_pos, double scale, float* cs, float* sn) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= n_pos * kNB) return;
    double s, c;
    sincos((double)(at / kNB) * f.f[at % kNB], &s, &c);
    cs[at] = (float)(scale * c);
    sn[at] = (float)(scale * s);
}

template <class T>
struct Elem;
template <>
struct Elem<__half> {
    static __device__ __forceinline__ void load8(const __half* p, float (&x)[8]) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);  // (plain loads: the rows may be rotated in place)
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            x[2 * i] = v.x;
            x[2 * i + 1] = v.y;
        }
    }
    static __device__ __forceinline__ void store8(__half* p, const float (&x)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = rope_h2(x[2 * i], x[2 * i + 1]);
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct Elem<float> {
    static __device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    static __device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};

struct RowsParams {
    RopeParams r;
    RowsView q, qo, k, ko;
    int n_q, n_k, t, share;  // share: heads a thread turns
    int64_t tokens;          // batch * t
    int inverse;
    int32_t* status;
};

constexpr int kRowThreads = 128;
constexpr int kRowLanes = 8;  // threads of a token and share
constexpr int kRowBatch = 2;  // rows a thread has in flight

template <class In, class Out>
__global__ void __launch_bounds__(kRowThreads) rope_rows_kernel(const __grid_constant__ RowsParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row = (int64_t)blockIdx.x * (kRowThreads / kRowLanes) + threadIdx.x / kRowLanes;
    if (row >= p.tokens) return;
    const int lane = threadIdx.x % kRowLanes;
    const int64_t b = row / p.t, i = row - b * p.t;
    int pos[kMaxAxes];
    if (!rope_positions(p.r, row, i, pos)) {
        if (lane == 0 && blockIdx.y == 0 && p.status) atomicOr(p.status, BGTQ_STATUS_ROPE_RANGE);
        return;
    }
    float c[8], s[8];
    {
        float c0[4], s0[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            rope_load4(p.r, pos, 8 * lane + 4 * k, c0, s0);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                c[4 * k + m] = c0[m];
                s[4 * k + m] = p.inverse ? -s0[m] : s0[m];
            }
        }
    }
    // layout 0: elements 8 lane .. and 64 + 8 lane ..; layout 1: 16 elements from 16 lane
    const int da = p.r.layout ? 16 * lane : 8 * lane, db = p.r.layout ? 16 * lane + 8 : 64 + 8 * lane;
    const int h0 = blockIdx.y * p.share, h1 = min(h0 + p.share, p.n_q + p.n_k);
    for (int h = h0; h < h1; h += kRowBatch) {
        float x[kRowBatch][2][8];
#pragma unroll
        for (int m = 0; m < kRowBatch; ++m) {
            const int hh = min(h + m, h1 - 1);
            const bool is_k = hh >= p.n_q;
            const RowsView& v = is_k ? p.k : p.q;
            const In* src = static_cast<const In*>(v.p) + b * v.sb + (int64_t)(is_k ? hh - p.n_q : hh) * v.sh + i * v.st;
            Elem<In>::load8(src + da, x[m][0]);
            Elem<In>::load8(src + db, x[m][1]);
        }
#pragma unroll
        for (int m = 0; m < kRowBatch; ++m) {
            const int hh = h + m;
            if (hh >= h1) break;
            if (p.r.layout == 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) rope_pair(x[m][0][e], x[m][1][e], c[e], s[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    rope_pair(x[m][0][2 * e], x[m][0][2 * e + 1], c[e], s[e]);
                    rope_pair(x[m][1][2 * e], x[m][1][2 * e + 1], c[4 + e], s[4 + e]);
                }
            }
            const bool is_k = hh >= p.n_q;
            const RowsView& v = is_k ? p.ko : p.qo;
            Out* dst = static_cast<Out*>(const_cast<void*>(v.p)) + b * v.sb + (int64_t)(is_k ? hh - p.n_q : hh) * v.sh + i * v.st;
            Elem<Out>::store8(dst + da, x[m][0]);
            Elem<Out>::store8(dst + db, x[m][1]);
        }
    }
}

template <class In, class Out>
cudaError_t go_rows(cudaStream_t s, RowsParams& p) {
    const int heads = p.n_q + p.n_k;
    const int64_t blocks = (p.tokens + kRowThreads / kRowLanes - 1) / (kRowThreads / kRowLanes);
    // heads shared out while the tokens alone leave the GPU's 152 SMs idle
    int parts = 1;
    while (parts < heads && blocks * parts < 8 * 152) parts *= 2;
    p.share = (heads + parts - 1) / parts;
    const unsigned gy = (unsigned)((heads + p.share - 1) / p.share);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, gy, 1);
    cfg.blockDim = dim3(kRowThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_rows_kernel<In, Out>, p);
}

template <class In>
cudaError_t go_rows_in(cudaStream_t s, RowsParams& p, int out_dtype) {
    switch (out_dtype) {
        case BGTQ_F16: return go_rows<In, __half>(s, p);
        case BGTQ_F32: return go_rows<In, float>(s, p);
        default: return go_rows<In, __nv_bfloat16>(s, p);
    }
}

}  // namespace

cudaError_t launch_rope_table(cudaStream_t s, const double* inv_freq, int64_t n_pos, double scale, float* cs, float* sn) {
    FreqTable f;
    for (int i = 0; i < kNB; ++i) f.f[i] = inv_freq[i];
    const int64_t blocks = (n_pos * kNB + 255) / 256;
    rope_table_kernel<<<(unsigned)blocks, 256, 0, s>>>(f, n_pos, scale, cs, sn);
    return cudaGetLastError();
}

cudaError_t launch_rope_rows(cudaStream_t s, const RopeParams& r, int batch, int t, const RowsView& q, const RowsView& q_out,
                             int n_q, const RowsView& k, const RowsView& k_out, int n_k, int in_dtype, int out_dtype,
                             int inverse, int32_t* status) {
    RowsParams p;
    p.r = r;
    p.q = q;
    p.qo = q_out;
    p.k = k;
    p.ko = k_out;
    p.n_q = n_q;
    p.n_k = n_k;
    p.t = t;
    p.tokens = (int64_t)batch * t;
    p.inverse = inverse;
    p.status = status;
    switch (in_dtype) {
        case BGTQ_F16: return go_rows_in<__half>(s, p, out_dtype);
        case BGTQ_F32: return go_rows_in<float>(s, p, out_dtype);
        default: return go_rows_in<__nv_bfloat16>(s, p, out_dtype);
    }
}

}  // namespace bgtq
