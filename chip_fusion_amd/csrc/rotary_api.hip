// C ABI of the norms and rotations of queries and keys (b2b_attn.h): checks,
// how a call is laid over workgroups, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "attn_plan.hpp"
#include "rotary_launch.hpp"

struct b2b_rotary_plan {
    int dtype, heads, kv_heads, dim, rotary, axes;
    bool norm, interleaved;
    float eps;
    double turns[64];
    uint8_t axis[64];
};

namespace {

using namespace b2b;

bool sizes_ok(const b2b_rotary_plan* p, int64_t rows) {
    return rows >= 0 && rows <= INT32_MAX / 2 && rows * (int64_t)(p->heads + 2 * p->kv_heads) <= INT32_MAX - 1024;
}

// Written rows: in place over their input, or apart from it, no two sharing an element.
bool written_ok(const b2b_rows_t& o, const b2b_rows_t& in, int64_t rows, int heads, int dim) {
    if (!out_ok(o, rows, heads, dim)) return false;
    if (o.data != in.data) return apart(extent(o, rows, heads, dim), {extent(in, rows, heads, dim)});
    return (rows <= 1 || o.row_stride == in.row_stride) && (heads <= 1 || o.head_stride == in.head_stride);
}

// Pages that are written: no two of their (page, row, head) share an element.
bool pages_apart(const b2b_pages_t& x, int64_t pages, int64_t size, int64_t heads, int64_t dim) {
    struct Dim {
        int64_t n, stride;
    } d[] = {{pages, x.page_stride}, {size, x.row_stride}, {heads, x.head_stride}};
    std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
    int64_t extent = dim;
    for (const Dim& y : d) {
        if (y.n <= 1) continue;
        if (y.stride < extent) return false;
        extent += (y.n - 1) * y.stride;
    }
    return true;
}

void fill(const b2b_rotary_plan* p, b2bk::RotaryArgs& a, int64_t rows, const b2b_rows_t& Q, const b2b_rows_t& K,
          const b2b_rows_t& Qo, const int32_t* positions, int64_t position_stride, const void* qw, const void* kw) {
    a.Q = dev(Q, p->dim);
    a.K = dev(K, p->dim);
    a.Qo = const_cast<void*>(Qo.data);
    a.ldqo = dev(Qo, p->dim).ld;
    a.hqo = Qo.head_stride;
    a.positions = positions;
    a.position_ld = position_stride;
    a.qw = qw;
    a.kw = kw;
    std::copy(p->turns, p->turns + 64, a.turns);
    std::copy(p->axis, p->axis + 64, a.axis);
    a.rows = (int32_t)rows;
    a.heads = p->heads;
    a.kv_heads = p->kv_heads;
    a.dim = p->dim;
    a.rotary = p->rotary;
    a.axes = p->axes;
    a.eps = p->eps;
}

bool weights_ok(const b2b_rotary_plan* p, const void* qw, const void* kw) {
    if (!p->norm) return !qw && !kw;
    return (uintptr_t)qw % 16 == 0 && (uintptr_t)kw % 16 == 0;
}

b2b_status_t go(const b2b_rotary_plan* p, b2bk::RotaryArgs& a, bool append, hipStream_t stream) {
    const int items = p->heads + (append ? 2 : 1) * p->kv_heads, groups = p->dim > 64 ? 16 : 32;
    // Rows a workgroup: its angles and its lanes' factors cost as much as some heads
    // do, so that a lane should take several, up to 10, as long as there are two
    // workgroups a compute unit (32 + 8 heads of 128, 16384 rows: 86 us with 1 row, 68
    // with 2, 64 with 4, 67 with 8; 16 + 4 of 64: 43, 32, 25 and 22; 2048 rows of the
    // first: 14.1, 13.0, 12.5, 17.3; 1024 rows: 8.1 with 1, 8.6 with 2).
    a.row_log = 0;
    if (a.rows >= 2048)
        while (2 << a.row_log <= b2bk::kRotaryRows && (2 << a.row_log) * items <= 10 * groups && a.rows >> (a.row_log + 1) >= 512)
            ++a.row_log;
    // Few rows: a head a lane, a row's heads over several workgroups (32 + 8 heads of
    // 128: 32 rows 5.2 us in one, 3.8 in three, 256 rows 5.5 and 4.7, 512 rows 6.3 and 7.3).
    const int share = a.rows <= 256 ? (int)ceil_div(items, groups) : 1;
    a.per_row.set(share);
    const int64_t grid = ceil_div(a.rows, (int64_t)1 << a.row_log) * share;
    if (grid > INT32_MAX) return B2B_ERROR_INVALID_VALUE;
    const RotaryLaunch L = p->dtype == B2B_DTYPE_F16 ? rotary_f16() : rotary_bf16();
    return L(a, {append, p->norm, p->interleaved}, (unsigned)grid, stream) == hipSuccess ? B2B_SUCCESS : B2B_ERROR_HIP;
}

}  // namespace

extern "C" {

b2b_status_t b2b_rotary_create(b2b_rotary_t* plan, b2b_dtype_t dtype, int32_t heads, int32_t kv_heads, int32_t head_dim,
                               int32_t rotary_dim, const double* freqs, const int32_t* axes_of, int32_t axes, float eps,
                               uint32_t flags) {
    if (!plan) return B2B_ERROR_INVALID_VALUE;
    *plan = nullptr;
    const bool norm = flags & B2B_ROTARY_NORM;
    if (heads < 1 || kv_heads < 1 || heads % kv_heads || heads > 65536 || head_dim < 1 || axes < 1 || axes > 4 ||
        (flags & ~(uint32_t)(B2B_ROTARY_NORM | B2B_ROTARY_INTERLEAVED)))
        return B2B_ERROR_INVALID_VALUE;
    if ((dtype != B2B_DTYPE_F16 && dtype != B2B_DTYPE_BF16) || head_dim % 8 || head_dim > 128)
        return B2B_ERROR_NOT_SUPPORTED;
    if (rotary_dim < 0 || rotary_dim > head_dim) return B2B_ERROR_INVALID_VALUE;
    if (rotary_dim % 8) return B2B_ERROR_NOT_SUPPORTED;
    if ((rotary_dim && !freqs) || (norm && !(eps >= 0.f && std::isfinite(eps)))) return B2B_ERROR_INVALID_VALUE;
    for (int i = 0; i < rotary_dim / 2; ++i)
        if (!std::isfinite(freqs[i]) || (axes_of && (axes_of[i] < 0 || axes_of[i] >= axes))) return B2B_ERROR_INVALID_VALUE;
    b2b_rotary_plan* p = new (std::nothrow) b2b_rotary_plan();
    if (!p) return B2B_ERROR_OUT_OF_MEMORY;
    p->dtype = dtype;
    p->heads = heads;
    p->kv_heads = kv_heads;
    p->dim = head_dim;
    p->rotary = rotary_dim;
    p->axes = axes;
    p->norm = norm;
    p->interleaved = flags & B2B_ROTARY_INTERLEAVED;
    p->eps = norm ? eps : 0.f;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        p->turns[i] = freqs[i] / 6.283185307179586476925;
        p->axis[i] = axes_of ? (uint8_t)axes_of[i] : 0;
    }
    *plan = p;
    return B2B_SUCCESS;
}

b2b_status_t b2b_rotary_run(b2b_rotary_t p, int64_t rows, b2b_rows_t Q, b2b_rows_t K, b2b_rows_t Qo, b2b_rows_t Ko,
                            const int32_t* positions, int64_t position_stride, const void* q_weight, const void* k_weight,
                            hipStream_t stream) {
    if (!p || !sizes_ok(p, rows) || !weights_ok(p, q_weight, k_weight)) return B2B_ERROR_INVALID_VALUE;
    if (!rows) return B2B_SUCCESS;
    if (!rows_ok(Q, rows, p->dim) || !rows_ok(K, rows, p->dim) || !written_ok(Qo, Q, rows, p->heads, p->dim) ||
        !written_ok(Ko, K, rows, p->kv_heads, p->dim))
        return B2B_ERROR_INVALID_VALUE;
    const Extent qo = extent(Qo, rows, p->heads, p->dim), ko = extent(Ko, rows, p->kv_heads, p->dim);
    if (!apart(qo, {ko, extent(K, rows, p->kv_heads, p->dim)}) || !apart(ko, {extent(Q, rows, p->heads, p->dim)}))
        return B2B_ERROR_INVALID_VALUE;
    if (p->rotary && (!positions || (p->axes > 1 && (position_stride < 0 || position_stride > kMaxFar))))
        return B2B_ERROR_INVALID_VALUE;
    b2bk::RotaryArgs a = {};
    fill(p, a, rows, Q, K, Qo, positions, position_stride, q_weight, k_weight);
    a.Ko = const_cast<void*>(Ko.data);
    a.ldko = dev(Ko, p->dim).ld;
    a.hko = Ko.head_stride;
    return go(p, a, false, stream);
}

b2b_status_t b2b_rotary_append(b2b_rotary_t p, int32_t seqs, int64_t rows, b2b_rows_t Q, b2b_rows_t K, b2b_rows_t V,
                               b2b_rows_t Qo, b2b_pages_t k_cache, b2b_pages_t v_cache, int32_t pages, int32_t page_size,
                               const int32_t* table, int32_t width, int64_t table_stride, const int32_t* lens,
                               const int32_t* cu, const int32_t* positions, int64_t position_stride, const void* q_weight,
                               const void* k_weight, hipStream_t stream) {
    if (!p || !sizes_ok(p, rows) || seqs < 0 || seqs > INT32_MAX / 2 || !weights_ok(p, q_weight, k_weight) || pages < 0 ||
        width < 0 || page_size < 1 || page_size > 1 << 20 || (!cu && rows != seqs))
        return B2B_ERROR_INVALID_VALUE;
    if (!rows || !seqs) return B2B_SUCCESS;
    if (!rows_ok(Q, rows, p->dim) || !rows_ok(K, rows, p->dim) || !rows_ok(V, rows, p->dim) ||
        !written_ok(Qo, Q, rows, p->heads, p->dim) || !lens)
        return B2B_ERROR_INVALID_VALUE;
    const Extent q = extent(Q, rows, p->heads, p->dim), k = extent(K, rows, p->kv_heads, p->dim),
                 v = extent(V, rows, p->kv_heads, p->dim), qo = extent(Qo, rows, p->heads, p->dim);
    if (!apart(qo, {k, v})) return B2B_ERROR_INVALID_VALUE;
    if (positions && p->axes > 1 && (position_stride < 0 || position_stride > kMaxFar)) return B2B_ERROR_INVALID_VALUE;
    if (pages && width) {
        if (!table || table_stride < 0 || table_stride > kMaxFar || (seqs > 1 && table_stride < width)) return B2B_ERROR_INVALID_VALUE;
        for (const b2b_pages_t* x : {&k_cache, &v_cache})
            if (!pages_ok(*x, pages) || !pages_apart(*x, pages, page_size, p->kv_heads, p->dim)) return B2B_ERROR_INVALID_VALUE;
        const Extent kc = extent(k_cache, pages, page_size, p->kv_heads, p->dim),
                     vc = extent(v_cache, pages, page_size, p->kv_heads, p->dim);
        if (!apart(kc, {q, k, v, qo, vc}) || !apart(vc, {q, k, v, qo})) return B2B_ERROR_INVALID_VALUE;
    }
    b2bk::RotaryArgs a = {};
    fill(p, a, rows, Q, K, Qo, positions, position_stride, q_weight, k_weight);
    a.V = dev(V, p->dim);
    a.ck = dev(k_cache);
    a.cv = dev(v_cache);
    a.page.set(page_size);
    a.table = table;
    a.table_ld = table_stride;
    a.lens = lens;
    a.cu = cu;
    a.seqs = seqs;
    a.pages = pages;
    a.width = pages ? width : 0;
    return go(p, a, true, stream);
}

b2b_status_t b2b_rotary_destroy(b2b_rotary_t plan) {
    delete plan;
    return B2B_SUCCESS;
}

}  // extern "C"
