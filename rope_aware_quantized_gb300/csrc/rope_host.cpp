// Entry points of the rotary operators and of the 4-bit cache: argument
// checks (the first ones read no device memory), then the launches.
#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "fp4.cuh"

namespace bgtq {

int check_rope(const bgtq_rope* r) {
    if (!r || !r->cos || !r->sin) return set_error(BGTQ_ERR_INVALID_ARG, "rope descriptor or one of its tables is NULL");
    if ((reinterpret_cast<uintptr_t>(r->cos) | reinterpret_cast<uintptr_t>(r->sin)) & 15)
        return set_error(BGTQ_ERR_INVALID_ARG, "cos and sin must be 16-byte aligned");
    if (r->n_pos < 1 || r->n_pos > INT32_MAX) return set_error(BGTQ_ERR_INVALID_ARG, "n_pos must be in [1, 2^31)");
    if (r->axes < 1 || r->axes > kMaxAxes) return set_error(BGTQ_ERR_INVALID_ARG, "axes must be in 1..4");
    if (r->layout != 0 && r->layout != 1) return set_error(BGTQ_ERR_INVALID_ARG, "rope layout must be 0 or 1");
    for (int i = 0; r->axis && i < kNB; ++i)
        if (r->axis[i] >= r->axes) return set_error(BGTQ_ERR_INVALID_ARG, "axis of block %d is %d of %d axes", i, r->axis[i], r->axes);
    return BGTQ_OK;
}

int check_rows(const bgtq_rows* r, const char* name, int batch, int heads, int64_t t, int elem, bool output) {
    if (!r || !r->data) return set_error(BGTQ_ERR_INVALID_ARG, "%s is NULL", name);
    const int64_t unit = 16 / elem;
    const int64_t ext[3] = {batch, heads, t}, str[3] = {r->stride_b, r->stride_h, r->stride_t};
    if (reinterpret_cast<uintptr_t>(r->data) & 15) return set_error(BGTQ_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
    for (int i = 0; i < 3; ++i) {
        if (ext[i] > 1 && (str[i] % unit)) return set_error(BGTQ_ERR_INVALID_ARG, "%s: strides must be multiples of 16 bytes", name);
        if (str[i] < 0) return set_error(BGTQ_ERR_INVALID_ARG, "%s: strides must be >= 0", name);
        if (ext[i] > 1 && str[i] > (INT64_C(1) << 52) / (ext[i] - 1))
            return set_error(BGTQ_ERR_INVALID_ARG, "%s: a stride is out of range", name);
    }
    if (!output) return BGTQ_OK;
    // rows of one dimension lie past the whole of the smaller ones
    int o[3] = {0, 1, 2};
    std::sort(o, o + 3, [&](int x, int y) { return str[x] < str[y]; });
    int64_t span = kD;
    for (int i : o) {
        if (ext[i] <= 1) continue;
        if (str[i] < span) return set_error(BGTQ_ERR_INVALID_ARG, "%s: its rows overlap one another", name);
        span += str[i] * (ext[i] - 1);
    }
    return BGTQ_OK;
}

}  // namespace bgtq

using namespace bgtq;

namespace {

int dtype_size(int d) { return d == BGTQ_F32 ? 4 : 2; }

// Bytes from the first to behind the last element of the rows.
int64_t extent(const bgtq_rows& r, int batch, int heads, int64_t t, int elem) {
    return (r.stride_b * (batch - 1) + r.stride_h * (heads - 1) + r.stride_t * (t - 1) + kD) * elem;
}

// Rows of two tensors with the same steps in memory: whether one row of each
// meets, i.e. some lo < delta + c0 s0 + c1 s1 + c2 s2 < hi with
// least[k] <= c[k] <= most[k] (s falling, steps of 0 left out).  A step is no
// shorter than the smaller ones' whole reach (outputs are checked for that), so
// few c fit in each.
struct Steps {
    int n = 0;
    int64_t s[3], least[3], most[3];
};
bool some_meet(const Steps& x, int k, int64_t delta, int64_t lo, int64_t hi) {
    if (k == x.n) return lo < delta && delta < hi;
    int64_t below = 0, above = 0;  // what the smaller steps can add
    for (int i = k + 1; i < x.n; ++i) {
        below += x.s[i] * -x.least[i];
        above += x.s[i] * x.most[i];
    }
    auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
    const int64_t first = std::max(x.least[k], floor_div(lo - above - delta, x.s[k]));
    const int64_t last = std::min(x.most[k], floor_div(hi + below - delta, x.s[k]) + 1);
    for (int64_t c = first; c <= last; ++c)
        if (some_meet(x, k + 1, delta + c * x.s[k], lo, hi)) return true;
    return false;
}

enum class Meet { kApart, kSame, kSome, kUnknown };
// Rows a (na heads) and b (nb): apart, the very same ones, some of them in one
// another, or (steps that differ within one another's extent) not told.
Meet rows_meet(const bgtq_rows& a, int na, int ea, const bgtq_rows& b, int nb, int eb, int batch, int64_t t) {
    const char *pa = static_cast<const char*>(a.data), *pb = static_cast<const char*>(b.data);
    if (pa + extent(a, batch, na, t, ea) <= pb || pb + extent(b, batch, nb, t, eb) <= pa) return Meet::kApart;
    const int64_t n[2][3] = {{batch, na, t}, {batch, nb, t}};
    const int64_t s[2][3] = {{a.stride_b * ea, a.stride_h * ea, a.stride_t * ea}, {b.stride_b * eb, b.stride_h * eb, b.stride_t * eb}};
    Steps x;
    for (int i = 0; i < 3; ++i) {
        if (n[0][i] == 1 && n[1][i] == 1) continue;
        if (n[0][i] > 1 && n[1][i] > 1 && s[0][i] != s[1][i]) return Meet::kUnknown;
        const int64_t step = n[1][i] > 1 ? s[1][i] : s[0][i];
        if (step == 0) return Meet::kUnknown;
        int k = x.n++;
        for (; k > 0 && x.s[k - 1] < step; --k) x.s[k] = x.s[k - 1], x.least[k] = x.least[k - 1], x.most[k] = x.most[k - 1];
        x.s[k] = step, x.least[k] = 1 - n[0][i], x.most[k] = n[1][i] - 1;
    }
    if (pa == pb && na == nb && ea == eb) return Meet::kSame;
    return some_meet(x, 0, pb - pa, (int64_t)-kD * eb, (int64_t)kD * ea) ? Meet::kSome : Meet::kApart;
}

// An output and its input: the same rows, or apart.
int check_in_place(const bgtq_rows& in, const bgtq_rows& out, const char* name, int batch, int heads, int64_t t, int di, int dt) {
    const Meet m = rows_meet(in, heads, dtype_size(di), out, heads, dtype_size(dt), batch, t);
    if (m == Meet::kApart || (m == Meet::kSame && di == dt)) return BGTQ_OK;
    return set_error(BGTQ_ERR_INVALID_ARG, "%s_out overlaps %s without being it", name, name);
}

int check_fp4(const bgtq_fp4_cache* c) {
    if (!c || !c->groups) return set_error(BGTQ_ERR_INVALID_ARG, "cache descriptor or its groups are NULL");
    if (reinterpret_cast<uintptr_t>(c->groups) & 15) return set_error(BGTQ_ERR_INVALID_ARG, "groups must be 16-byte aligned");
    if (c->capacity < kGroup || c->capacity % kGroup || c->capacity > (1 << 30))
        return set_error(BGTQ_ERR_INVALID_ARG, "capacity must be a multiple of 16 in [16, 2^30]");
    if (c->n_heads < 1 || c->n_heads > 4096) return set_error(BGTQ_ERR_INVALID_ARG, "n_heads must be in 1..4096");
    if (c->page_table) {
        const int64_t P = c->page_tokens;
        if (P < 16 || P > (1 << 20) || (P & (P - 1)))
            return set_error(BGTQ_ERR_INVALID_ARG, "page_tokens must be a power of two in [16, 2^20]");
        if (c->max_pages < 1 || c->n_pages < 1 || c->n_pages > INT32_MAX)
            return set_error(BGTQ_ERR_INVALID_ARG, "max_pages and n_pages must be >= 1 (n_pages < 2^31)");
        if (c->max_pages > c->capacity || c->capacity != c->max_pages * P)
            return set_error(BGTQ_ERR_INVALID_ARG, "a paged cache needs capacity == max_pages * page_tokens");
        if (reinterpret_cast<uintptr_t>(c->page_table) & 3)
            return set_error(BGTQ_ERR_INVALID_ARG, "page_table must be 4-byte aligned");
    }
    return BGTQ_OK;
}

// k, v and pos_start of an append.
int check_new(const bgtq_rope* rope, const int32_t* pos, const bgtq_rows* k, const bgtq_rows* v, int batch, int heads, int t_new,
              const int32_t* pos_start) {
    if (rope) {
        const int rc = check_rope(rope);
        if (rc) return rc;
    } else if (pos) {
        return set_error(BGTQ_ERR_INVALID_ARG, "pos without rope");
    }
    if (!pos_start) return set_error(BGTQ_ERR_INVALID_ARG, "pos_start is NULL");
    int rc = check_rows(k, "k", batch, heads, t_new, 2, false);
    if (rc) return rc;
    return check_rows(v, "v", batch, heads, t_new, 2, false);
}

}  // namespace

extern "C" {

int bgtq_rope_table(void* stream, const double* inv_freq, int64_t n_pos, double scale, float* cs, float* sn) {
    if (!inv_freq || !cs || !sn) return set_error(BGTQ_ERR_INVALID_ARG, "NULL pointer");
    if (n_pos < 1 || n_pos > INT32_MAX) return set_error(BGTQ_ERR_INVALID_ARG, "n_pos must be in [1, 2^31)");
    if ((reinterpret_cast<uintptr_t>(cs) | reinterpret_cast<uintptr_t>(sn)) & 15)
        return set_error(BGTQ_ERR_INVALID_ARG, "cos and sin must be 16-byte aligned");
    if (!std::isfinite(scale)) return set_error(BGTQ_ERR_INVALID_ARG, "scale must be finite");
    for (int i = 0; i < kNB; ++i)
        if (!std::isfinite(inv_freq[i])) return set_error(BGTQ_ERR_INVALID_ARG, "inv_freq[%d] is not finite", i);
    const cudaError_t e = launch_rope_table((cudaStream_t)stream, inv_freq, n_pos, scale, cs, sn);
    if (e != cudaSuccess) return set_error(BGTQ_ERR_CUDA, "rope_table launch: %s", cudaGetErrorString(e));
    return BGTQ_OK;
}

int bgtq_rope_rows(void* stream, const bgtq_rope* rope, const int32_t* pos, int batch, int t, const bgtq_rows* q,
                   const bgtq_rows* q_out, int n_q, const bgtq_rows* k, const bgtq_rows* k_out, int n_k, int in_dtype,
                   int out_dtype, int inverse, int32_t* status) {
    int rc = check_rope(rope);
    if (rc) return rc;
    if (batch < 0 || t < 0 || n_q < 0 || n_k < 0) return set_error(BGTQ_ERR_INVALID_ARG, "batch, t and head counts must be >= 0");
    if (n_q > 65535 || n_k > 65535) return set_error(BGTQ_ERR_UNSUPPORTED, "at most 65535 heads");
    if (in_dtype < 0 || in_dtype > 2 || out_dtype < 0 || out_dtype > 2)
        return set_error(BGTQ_ERR_INVALID_ARG, "dtypes must be BGTQ_F16, BGTQ_F32 or BGTQ_BF16");
    if (inverse != 0 && inverse != 1) return set_error(BGTQ_ERR_INVALID_ARG, "inverse must be 0 or 1");
    if (batch == 0 || t == 0 || n_q + n_k == 0) return BGTQ_OK;
    if (!pos) return set_error(BGTQ_ERR_INVALID_ARG, "pos is NULL");
    if ((uint64_t)batch * (uint64_t)t >= (1ull << 31)) return set_error(BGTQ_ERR_UNSUPPORTED, "batch * t must stay below 2^31");
    const int ei = dtype_size(in_dtype), eo = dtype_size(out_dtype);
    RowsView none = {nullptr, 0, 0, 0}, qi = none, qo = none, ki = none, ko = none;
    if (n_q) {
        if ((rc = check_rows(q, "q", batch, n_q, t, ei, false)) || (rc = check_rows(q_out, "q_out", batch, n_q, t, eo, true))) return rc;
        qi = make_rows(*q), qo = make_rows(*q_out);
    }
    if (n_k) {
        if ((rc = check_rows(k, "k", batch, n_k, t, ei, false)) || (rc = check_rows(k_out, "k_out", batch, n_k, t, eo, true))) return rc;
        ki = make_rows(*k), ko = make_rows(*k_out);
    }
    if (n_q && n_k) {
        const Meet m = rows_meet(*q_out, n_q, eo, *k_out, n_k, eo, batch, t);
        if (m == Meet::kSome || m == Meet::kSame) return set_error(BGTQ_ERR_INVALID_ARG, "q_out and k_out overlap");
    }
    if (n_q && (rc = check_in_place(*q, *q_out, "q", batch, n_q, t, in_dtype, out_dtype))) return rc;
    if (n_k && (rc = check_in_place(*k, *k_out, "k", batch, n_k, t, in_dtype, out_dtype))) return rc;
    const cudaError_t e = launch_rope_rows((cudaStream_t)stream, make_rope(rope, pos, (int64_t)batch * t), batch, t, qi, qo, n_q,
                                           ki, ko, n_k, in_dtype, out_dtype, inverse, status);
    if (e != cudaSuccess) return set_error(BGTQ_ERR_CUDA, "rope_rows launch: %s", cudaGetErrorString(e));
    return BGTQ_OK;
}

int bgtq_rope_append(const bgtq_plan* p, void* stream, const bgtq_rope* rope, const int32_t* pos, const bgtq_rows* k,
                     const bgtq_rows* v, int batch, int t_new, const int32_t* pos_start, const bgtq_cache* c, int32_t* status) {
    if (!p) return set_error(BGTQ_ERR_INVALID_ARG, "plan is NULL");
    int rc = check_cache(p, c);
    if (rc) return rc;
    if (!rope) return set_error(BGTQ_ERR_INVALID_ARG, "rope is NULL");
    if (batch < 0 || t_new < 0) return set_error(BGTQ_ERR_INVALID_ARG, "batch and t_new must be >= 0");
    if (batch > 32767) return set_error(BGTQ_ERR_UNSUPPORTED, "at most 32767 sequences per call");
    if (batch == 0 || t_new == 0) return check_rope(rope);
    if ((rc = check_new(rope, pos, k, v, batch, p->H, t_new, pos_start))) return rc;
    if (rope->layout != p->rope_layout)
        return set_error(BGTQ_ERR_INVALID_ARG, "the rope's layout is %d, the plan's %d", rope->layout, p->rope_layout);
    if ((rc = check_plan_here(p))) return rc;
    const cudaError_t e = launch_rope_append(*p, (cudaStream_t)stream, make_rope(rope, pos, (int64_t)batch * t_new), make_rows(*k),
                                             make_rows(*v), batch, t_new, pos_start, *c, status);
    if (e != cudaSuccess) return set_error(BGTQ_ERR_CUDA, "rope_append launch: %s", cudaGetErrorString(e));
    return BGTQ_OK;
}

int bgtq_fp4_cache_bytes(int H, int batch, int64_t capacity, size_t* bytes) {
    if (!bytes) return set_error(BGTQ_ERR_INVALID_ARG, "NULL pointer");
    if (H < 1 || H > 4096 || batch < 0 || capacity < 0 || capacity % kGroup || capacity > (1 << 30))
        return set_error(BGTQ_ERR_INVALID_ARG, "bad head count, batch or capacity (a multiple of 16, at most 2^30)");
    if (capacity && (uint64_t)batch * H > (uint64_t)INT64_MAX / kGroupBytes / (uint64_t)(capacity / kGroup))
        return set_error(BGTQ_ERR_UNSUPPORTED, "the groups' bytes do not fit 64 bits");
    *bytes = (size_t)batch * H * (size_t)(capacity / kGroup) * kGroupBytes;
    return BGTQ_OK;
}

int bgtq_fp4_append(void* stream, const bgtq_rope* rope, const int32_t* pos, const bgtq_rows* k, const bgtq_rows* v, int batch,
                    int t_new, const int32_t* pos_start, const bgtq_fp4_cache* c, int32_t* status) {
    int rc = check_fp4(c);
    if (rc) return rc;
    if (batch < 0 || t_new < 0) return set_error(BGTQ_ERR_INVALID_ARG, "batch and t_new must be >= 0");
    if (batch > 65535) return set_error(BGTQ_ERR_UNSUPPORTED, "at most 65535 sequences per call");
    if (batch == 0 || t_new == 0) return BGTQ_OK;
    if ((rc = check_new(rope, pos, k, v, batch, c->n_heads, t_new, pos_start))) return rc;
    if (fp4_append_blocks(fp4_append_groups(t_new, c->capacity), c->n_heads) > INT32_MAX)
        return set_error(BGTQ_ERR_UNSUPPORTED, "t_new / 64 * heads must stay below 2^31");
    const cudaError_t e = launch_fp4_append((cudaStream_t)stream, make_rope(rope, pos, (int64_t)batch * t_new), make_rows(*k),
                                            make_rows(*v), batch, t_new, pos_start, *c, status);
    if (e != cudaSuccess) return set_error(BGTQ_ERR_CUDA, "fp4_append launch: %s", cudaGetErrorString(e));
    return BGTQ_OK;
}

int bgtq_fp4_attn_workspace(int H, int group, int batch, int t, int64_t max_len, size_t* bytes) {
    if (!bytes) return set_error(BGTQ_ERR_INVALID_ARG, "NULL pointer");
    if (H < 1 || H > 4096 || group < 1 || group > 8) return set_error(BGTQ_ERR_INVALID_ARG, "head counts: 1..4096 KV heads, groups of 1..8");
    if (batch < 0 || t < 0 || max_len < 0 || max_len > (1 << 30))
        return set_error(BGTQ_ERR_INVALID_ARG, "batch, t and max_len must be >= 0 (max_len at most 2^30)");
    *bytes = fp4_attn_workspace_bytes(H, group, batch, t, max_len);
    return BGTQ_OK;
}

int bgtq_fp4_attn(void* stream, const bgtq_rope* rope, const int32_t* pos, const bgtq_rows* q, int group, int batch, int t,
                  const bgtq_fp4_cache* c, const int32_t* seq_lens, int64_t max_len, void* out, int out_dtype, float scale,
                  void* ws, size_t ws_bytes, int32_t* status) {
    int rc = check_fp4(c);
    if (rc) return rc;
    if (batch < 0 || t < 0 || max_len < 0) return set_error(BGTQ_ERR_INVALID_ARG, "batch, t and max_len must be >= 0");
    if (group < 1 || group > 8) return set_error(BGTQ_ERR_INVALID_ARG, "group must be in 1..8");
    if (out_dtype != 0 && out_dtype != 1) return set_error(BGTQ_ERR_INVALID_ARG, "out_dtype must be 0 (half) or 1 (float)");
    // (a larger one could take logits past the kernels' first reference, -1e30: |q.k| < 2^39)
    if (!(scale > 0.0f) || !(scale <= 1099511627776.0f)) return set_error(BGTQ_ERR_INVALID_ARG, "softmax_scale must be in (0, 2^40]");
    if (batch > 65535 || (int64_t)batch * c->n_heads > 65535)
        return set_error(BGTQ_ERR_UNSUPPORTED, "at most 65535 sequences x KV heads per call");
    if (batch == 0 || t == 0) return BGTQ_OK;
    if (rope) {
        if ((rc = check_rope(rope))) return rc;
    } else if (pos) {
        return set_error(BGTQ_ERR_INVALID_ARG, "pos without rope");
    }
    if ((rc = check_rows(q, "q", batch, c->n_heads * group, t, 2, false))) return rc;
    if (!seq_lens || !out || !ws) return set_error(BGTQ_ERR_INVALID_ARG, "NULL pointer");
    if (reinterpret_cast<uintptr_t>(out) & 15) return set_error(BGTQ_ERR_INVALID_ARG, "out must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(ws) & 255) return set_error(BGTQ_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    max_len = std::min(max_len, c->capacity);
    if ((uint64_t)batch * c->n_heads * group * (uint64_t)t + 256 >= (1ull << 31))
        return set_error(BGTQ_ERR_UNSUPPORTED, "batch * query heads * t + 256 must stay below 2^31");
    if ((uint64_t)batch * c->n_heads * (uint64_t)(max_len / kGroup + 1) >= (1ull << 30))
        return set_error(BGTQ_ERR_UNSUPPORTED, "batch * heads * max_len must stay below 2^34");
    const size_t need = fp4_attn_workspace_bytes(c->n_heads, group, batch, t, max_len);
    if (ws_bytes < need) return set_error(BGTQ_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
    Fp4Attn a;
    a.rope = make_rope(rope, pos, (int64_t)batch * t);
    a.q = make_rows(*q);
    a.map = make_fp4_map(*c, batch, status);
    a.seq_lens = seq_lens;
    a.cap = c->capacity;
    a.max_len = max_len;
    a.batch = batch;
    a.t = t;
    a.group = group;
    a.out = out;
    a.out_dtype = out_dtype;
    a.scale = scale;
    a.ws = ws;
    a.status = status;
    const cudaError_t e = launch_fp4_attn((cudaStream_t)stream, a);
    if (e != cudaSuccess) return set_error(BGTQ_ERR_CUDA, "fp4_attn launch: %s", cudaGetErrorString(e));
    return BGTQ_OK;
}

int bgtq_fp4_dequant(void* stream, const bgtq_fp4_cache* c, int batch, int b, int head, int64_t t0, int64_t t1, float* k_out,
                     float* v_out) {
    const int rc = check_fp4(c);
    if (rc) return rc;
    if (b < 0 || b >= batch || head < 0 || head >= c->n_heads) return set_error(BGTQ_ERR_INVALID_ARG, "sequence or head out of range");
    if (t0 < 0 || t1 < t0 || t1 > c->capacity) return set_error(BGTQ_ERR_INVALID_ARG, "positions out of range");
    if (t0 == t1 || (!k_out && !v_out)) return BGTQ_OK;
    const cudaError_t e = launch_fp4_dequant((cudaStream_t)stream, *c, batch, b, head, t0, t1, k_out, v_out);
    if (e != cudaSuccess) return set_error(BGTQ_ERR_CUDA, "fp4_dequant launch: %s", cudaGetErrorString(e));
    return BGTQ_OK;
}

}  // extern "C"
