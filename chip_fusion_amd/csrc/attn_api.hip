// C ABI of the attention operators (b2b_attn.h): checks, how a call is split
// over workgroups, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <new>

#include "attn_plan.hpp"
#include "linear_attn_launch.hpp"

struct b2b_linear_attn_plan {
    int dtype, heads, kv_heads, dim;
    float scale;
};

namespace {

using namespace b2b;

// How a call with this many query rows a key head (in all, and a sequence on
// average) and keys is laid over workgroups.
struct Split {
    int64_t tiles;     // row tiles at most
    int splits;        // parts of the keys
};
Split plan_tiles(const b2b_attn_plan* p, int64_t seqs, int64_t rows, int64_t keys) {
    const int64_t fill = 512;      // workgroups: two a compute unit
    const int64_t group = p->heads / p->kv_heads;
    Split s;
    s.tiles = rows * group / b2b::kAttnRows + seqs;
    const int64_t wgs = s.tiles * p->kv_heads, each = keys / seqs;
    // Parts of the keys.  Too few workgroups for `fill`: parts of 256 keys or
    // more.  Where most keys come before the rows (pieces of prompts), contexts
    // differ and one workgroup's may be twice the average while all of them run
    // at once: up to two workgroups a slot, parts of 800 or more, so that
    // writing and joining partial results stays below what the balance gains
    // (2500 rows behind 0..4096 keys, 24 heads of 96: 106 us whole, 85 in two
    // parts, 88 in three, 111 in four; 8001 rows of 32 heads, their own keys only: 63
    // us whole, 165 in two).
    int64_t parts = std::min(fill / wgs, each / 256);
    if (keys >= 2 * rows) parts = std::max(parts, std::min(2 * fill / wgs, each / 800));
    s.splits = (int)std::max<int64_t>(1, std::min<int64_t>(parts, 64));
    return s;
}
// A prefix: 1.5 workgroups a compute unit, beside those of the requests' own
// keys (128 requests behind 32768 tokens, 32 heads of 128: 141 us at 1, 124 at
// 1.5, 128 at 2, 146 at 3), and parts of 256 keys or more, of a few rows 64
// (partial results cost little then: 3 requests of 8 heads behind 300 tokens
// take 6.2 us on the device instead of 10.6; 32 requests of 32 heads behind 4097
// took 26 us in parts of 128, 20 in parts of 256 and 23 in parts of 512).
Split plan_prefix(const b2b_attn_plan* p, int64_t batch, int64_t prefix) {
    Split s;
    s.tiles = ceil_div(batch * (p->heads / p->kv_heads), b2b::kAttnRows);
    const int64_t least = batch * p->heads <= 512 ? 64 : 256;
    s.splits = (int)std::max<int64_t>(1, std::min<int64_t>({384 / (s.tiles * p->kv_heads), prefix / least, 64}));
    return s;
}
// the many-requests kernel's parts of a request's own keys
int plan_own(const b2b_attn_plan* p, int64_t batch, int64_t own) {
    const int64_t wgs = batch * p->kv_heads * ceil_div(p->heads / p->kv_heads, 32);
    return (int)std::max<int64_t>(1, std::min<int64_t>({256 / wgs, own / 256, 64}));
}

size_t part_bytes(const b2b_attn_plan* p, int64_t slots, int64_t rows) {
    return (size_t)slots * rows * p->heads * (p->dim + 1) * 4;
}

const b2b::AttnLaunch& launchers(const b2b_attn_plan* p) {
    return p->dtype == B2B_DTYPE_F16 ? b2b::attn_f16() : b2b::attn_bf16();
}

}  // namespace

b2b_status_t b2b::create_attn(b2b_attn_t* plan, b2b_dtype_t dtype, int32_t heads, int32_t kv_heads, int32_t head_dim,
                              float scale, bool causal, int32_t window, int32_t sinks, int32_t page) {
    if (heads < 1 || kv_heads < 1 || heads % kv_heads || heads > 65536 || head_dim < 1) return B2B_ERROR_INVALID_VALUE;
    if (!(scale >= 0.f) || !std::isfinite(scale * b2bk::kLog2e)) return B2B_ERROR_INVALID_VALUE;
    if ((dtype != B2B_DTYPE_F16 && dtype != B2B_DTYPE_BF16) || head_dim % 8 || head_dim > 128)
        return B2B_ERROR_NOT_SUPPORTED;
    b2b_attn_plan* p = new (std::nothrow) b2b_attn_plan();
    if (!p) return B2B_ERROR_OUT_OF_MEMORY;
    p->dtype = dtype;
    p->heads = heads;
    p->kv_heads = kv_heads;
    p->dim = head_dim;
    p->scale = scale > 0.f ? scale : (float)(1.0 / std::sqrt((double)head_dim));
    p->causal = causal;
    p->window = window;
    p->sinks = sinks;
    p->page = page;
    *plan = p;
    return B2B_SUCCESS;
}

extern "C" {

b2b_status_t b2b_attn_create(b2b_attn_t* plan, b2b_dtype_t dtype, int32_t heads, int32_t kv_heads, int32_t head_dim,
                             float scale, uint32_t flags) {
    if (!plan) return B2B_ERROR_INVALID_VALUE;
    *plan = nullptr;
    if (flags & ~(uint32_t)B2B_ATTN_CAUSAL) return B2B_ERROR_INVALID_VALUE;
    return create_attn(plan, dtype, heads, kv_heads, head_dim, scale, (flags & B2B_ATTN_CAUSAL) != 0, 0, 0, 0);
}

b2b_status_t b2b_attn_destroy(b2b_attn_t plan) {
    delete plan;
    return B2B_SUCCESS;
}

b2b_status_t b2b_attn_workspace(b2b_attn_t p, int32_t seqs, int64_t rows, int64_t keys, size_t* bytes) {
    if (!p || !bytes || p->page || !sizes_ok(p, seqs, rows, keys)) return B2B_ERROR_INVALID_VALUE;
    if (p->window) return window_workspace(p, seqs, rows, keys, bytes);
    *bytes = 0;
    if (!seqs || !rows) return B2B_SUCCESS;
    const Split s = plan_tiles(p, seqs, rows, keys);
    if (s.splits > 1) *bytes = part_bytes(p, s.splits, rows);
    return B2B_SUCCESS;
}

b2b_status_t b2b_attn_run(b2b_attn_t p, int32_t seqs, int64_t rows, int64_t keys, b2b_rows_t Q, b2b_rows_t K,
                          b2b_rows_t V, b2b_rows_t O, const int32_t* cu_q, const int32_t* cu_k, float* lse,
                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!p || p->page || !sizes_ok(p, seqs, rows, keys)) return B2B_ERROR_INVALID_VALUE;
    if (!seqs || !rows) return B2B_SUCCESS;
    const int dim = p->dim;
    if (!rows_ok(Q, rows, dim) || !out_ok(O, rows, p->heads, dim) || !cu_q || !cu_k) return B2B_ERROR_INVALID_VALUE;
    if (keys && (!rows_ok(K, keys, dim) || !rows_ok(V, keys, dim))) return B2B_ERROR_INVALID_VALUE;
    if (O.data == Q.data || O.data == K.data || O.data == V.data || (uintptr_t)lse % 4) return B2B_ERROR_INVALID_VALUE;
    if (p->window)
        return window_run(p, seqs, rows, keys, Q, K, V, O, cu_q, cu_k, lse, workspace, workspace_bytes, stream);
    const Split s = plan_tiles(p, seqs, rows, keys);
    size_t need = s.splits > 1 ? part_bytes(p, s.splits, rows) : 0;
    if (need && (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < need)) return B2B_ERROR_INVALID_VALUE;
    b2bk::AttnArgs a = {};
    base_args(p, a);
    a.Q = dev(Q, dim);
    a.K = dev(K, dim);
    a.V = dev(V, dim);
    a.O = const_cast<void*>(O.data);
    a.ldo = O.row_stride;
    a.hso = O.head_stride;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.rows = rows;
    a.keys = keys;
    a.lse = lse;
    a.seqs = seqs;
    a.causal = p->causal;
    a.splits.set(s.splits);
    a.tiles = (int32_t)s.tiles;
    a.part = (float*)workspace;
    a.part_lse = a.part + (size_t)s.splits * rows * p->heads * dim;
    const int64_t grid = s.tiles * p->kv_heads * s.splits;
    if (grid > INT32_MAX) return B2B_ERROR_INVALID_VALUE;
    const b2b::AttnLaunch& L = launchers(p);
    if (L.tile(a, s.splits > 1, (unsigned)grid, stream) != hipSuccess) return B2B_ERROR_HIP;
    if (s.splits > 1 && L.join(a, s.splits, stream) != hipSuccess) return B2B_ERROR_HIP;
    return B2B_SUCCESS;
}

b2b_status_t b2b_prefix_attn_workspace(b2b_attn_t p, int32_t batch, int64_t prefix, int64_t own, size_t* bytes) {
    if (!p || !bytes || !sizes_ok(p, batch, batch, prefix) || own < 0 || own > INT32_MAX / 2)
        return B2B_ERROR_INVALID_VALUE;
    *bytes = 0;
    if (!batch) return B2B_SUCCESS;
    const int64_t slots = (prefix ? plan_prefix(p, batch, prefix).splits : 0) + (own ? plan_own(p, batch, own) : 0);
    *bytes = part_bytes(p, slots, batch);
    return B2B_SUCCESS;
}

b2b_status_t b2b_prefix_attn_run(b2b_attn_t p, int32_t batch, int64_t prefix, int64_t own, b2b_rows_t Q,
                                 b2b_rows_t Kp, b2b_rows_t Vp, b2b_rows_t K, int64_t k_stride, b2b_rows_t V,
                                 int64_t v_stride, const int32_t* lens, b2b_rows_t O, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    size_t need = 0;
    if (!p || p->causal) return B2B_ERROR_INVALID_VALUE;      // (nor a window or pages, which are causal)
    const b2b_status_t st = b2b_prefix_attn_workspace(p, batch, prefix, own, &need);
    if (st != B2B_SUCCESS) return st;
    if (!batch) return B2B_SUCCESS;
    const int dim = p->dim;
    if (!rows_ok(Q, batch, dim) || !out_ok(O, batch, p->heads, dim) || O.data == Q.data) return B2B_ERROR_INVALID_VALUE;
    if (prefix && (!rows_ok(Kp, prefix, dim) || !rows_ok(Vp, prefix, dim) || O.data == Kp.data || O.data == Vp.data))
        return B2B_ERROR_INVALID_VALUE;
    if (own && (!rows_ok(K, own, dim) || !rows_ok(V, own, dim) || !lens || k_stride < 0 || v_stride < 0 ||
                k_stride > kMaxFar || v_stride > kMaxFar || k_stride % 8 || v_stride % 8 || O.data == K.data || O.data == V.data))
        return B2B_ERROR_INVALID_VALUE;
    if (need && (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < need)) return B2B_ERROR_INVALID_VALUE;
    const b2b::AttnLaunch& L = launchers(p);
    b2bk::AttnArgs a = {};
    base_args(p, a);
    a.Q = dev(Q, dim);
    a.O = const_cast<void*>(O.data);
    a.ldo = O.row_stride;
    a.hso = O.head_stride;
    a.rows = batch;
    const Split s = prefix ? plan_prefix(p, batch, prefix) : Split{0, 0};
    const int own_parts = own ? plan_own(p, batch, own) : 0, slots = s.splits + own_parts;
    a.part = (float*)workspace;
    a.part_lse = a.part + (size_t)slots * batch * p->heads * dim;
    const int64_t grid_p = s.tiles * p->kv_heads * s.splits;
    const int64_t row_tiles = ceil_div(p->heads / p->kv_heads, 32);
    const int64_t grid_o = (int64_t)batch * row_tiles * p->kv_heads * own_parts;
    if (grid_p + grid_o > INT32_MAX) return B2B_ERROR_INVALID_VALUE;
    a.splits.set(std::max(s.splits, 1));
    a.tiles = (int32_t)s.tiles;
    a.seqs = 1;
    b2bk::AttnArgs o = a;
    if (prefix) {
        a.K = dev(Kp, dim);
        a.V = dev(Vp, dim);
        a.keys = prefix;
    }
    if (own) {
        o.K = dev(K, dim);
        o.V = dev(V, dim);
        o.lens = lens;
        o.k_stride = k_stride;
        o.v_stride = v_stride;
        o.keys = own;
        o.seqs = batch;
        o.splits.set(own_parts);
        o.slot0 = s.splits;
        o.tiles = (int32_t)row_tiles;
    }
    if (grid_p + grid_o && L.prefix(a, o, (unsigned)grid_p, (unsigned)grid_o, stream) != hipSuccess) return B2B_ERROR_HIP;
    return L.join(a, slots, stream) == hipSuccess ? B2B_SUCCESS : B2B_ERROR_HIP;
}

b2b_status_t b2b_linear_attn_create(b2b_linear_attn_t* plan, b2b_dtype_t dtype, int32_t heads, int32_t kv_heads,
                                    int32_t head_dim, float scale) {
    if (!plan) return B2B_ERROR_INVALID_VALUE;
    *plan = nullptr;
    if (heads < 1 || kv_heads < 1 || heads % kv_heads || heads > 65536 || head_dim < 1) return B2B_ERROR_INVALID_VALUE;
    if (!(scale >= 0.f) || !std::isfinite(scale)) return B2B_ERROR_INVALID_VALUE;
    if ((dtype != B2B_DTYPE_F16 && dtype != B2B_DTYPE_BF16) || (head_dim != 64 && head_dim != 128))
        return B2B_ERROR_NOT_SUPPORTED;
    b2b_linear_attn_plan* p = new (std::nothrow) b2b_linear_attn_plan();
    if (!p) return B2B_ERROR_OUT_OF_MEMORY;
    p->dtype = dtype;
    p->heads = heads;
    p->kv_heads = kv_heads;
    p->dim = head_dim;
    p->scale = scale > 0.f ? scale : (float)(1.0 / std::sqrt((double)head_dim));
    *plan = p;
    return B2B_SUCCESS;
}

b2b_status_t b2b_linear_attn_destroy(b2b_linear_attn_t plan) {
    delete plan;
    return B2B_SUCCESS;
}

}  // extern "C"

namespace {

// Tokens of a segment.  A workgroup, one a compute unit, takes a sequence's
// head; where those are fewer than compute units, sequences are cut into
// segments of 512 tokens or more, at the price of reading K and V twice (8200
// tokens in 9 sequences of 32 heads, 288 workgroups: 82 us whole, 124 to 126
// in segments of 512 to 1024; one of 32768 with 16 heads, fp16: 1364 us whole,
// 290 in 8 segments, 195 in 16, 207 in 32, 234 in 64).
int64_t lin_segment(const b2b_linear_attn_plan* p, int64_t seqs, int64_t rows) {
    const int64_t want = std::max(1, 256 / p->heads);
    if (seqs >= want) return INT32_MAX;
    return std::max<int64_t>(512, ceil_div(ceil_div(rows, want), 64) * 64);
}
bool lin_split(const b2b_linear_attn_plan* p, int64_t seqs, int64_t rows, int64_t* seg) {
    *seg = lin_segment(p, seqs, rows);
    return rows > *seg;
}
bool lin_sizes_ok(const b2b_linear_attn_plan* p, int64_t seqs, int64_t rows) {
    return seqs >= 0 && rows >= 0 && rows <= INT32_MAX / 2 && seqs <= INT32_MAX / 2 &&
           (rows + seqs) * (int64_t)p->heads <= INT32_MAX / 16;
}
size_t lin_bytes(const b2b_linear_attn_plan* p, int64_t seqs, int64_t rows) {
    int64_t seg;
    if (!seqs || !lin_split(p, seqs, rows, &seg)) return 0;
    return (size_t)(rows / seg + seqs) * p->heads * p->dim * p->dim * 4;
}
b2bk::LinArgs lin_args(const b2b_linear_attn_plan* p, const b2b_rows_t& Q, const b2b_rows_t& K, const b2b_rows_t& V,
                       const b2b_rows_t& O) {
    b2bk::LinArgs a = {};
    a.Q = dev(Q, p->dim);
    a.K = dev(K, p->dim);
    a.V = dev(V, p->dim);
    a.O = const_cast<void*>(O.data);
    a.ldo = dev(O, p->dim).ld;      // a chunk's stores step by it past a single row too
    a.hso = O.head_stride;
    a.heads = p->heads;
    a.kv_heads = p->kv_heads;
    a.group = p->heads / p->kv_heads;
    a.scale = p->scale;
    return a;
}
bool lin_operands_ok(const b2b_linear_attn_plan* p, int64_t rows, const b2b_rows_t& Q, const b2b_rows_t& K,
                     const b2b_rows_t& V, const b2b_rows_t& O) {
    return rows_ok(Q, rows, p->dim) && rows_ok(K, rows, p->dim) && rows_ok(V, rows, p->dim) &&
           out_ok(O, rows, p->heads, p->dim) && O.data != Q.data && O.data != K.data && O.data != V.data;
}

}  // namespace

extern "C" {

b2b_status_t b2b_linear_attn_workspace(b2b_linear_attn_t p, int32_t seqs, int64_t rows, size_t* bytes) {
    if (!p || !bytes || !lin_sizes_ok(p, seqs, rows)) return B2B_ERROR_INVALID_VALUE;
    *bytes = lin_bytes(p, seqs, rows);
    return B2B_SUCCESS;
}

b2b_status_t b2b_linear_attn_run(b2b_linear_attn_t p, int32_t seqs, int64_t rows, b2b_rows_t Q, b2b_rows_t K,
                                 b2b_rows_t V, b2b_rows_t O, const float* log_decay, const int32_t* cu,
                                 const float* state_in, float* state_out, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream) {
    if (!p || !lin_sizes_ok(p, seqs, rows)) return B2B_ERROR_INVALID_VALUE;
    if (!seqs) return B2B_SUCCESS;
    if (!log_decay || !cu || (uintptr_t)state_in % 16 || (uintptr_t)state_out % 16) return B2B_ERROR_INVALID_VALUE;
    if (rows && !lin_operands_ok(p, rows, Q, K, V, O)) return B2B_ERROR_INVALID_VALUE;
    const size_t need = lin_bytes(p, seqs, rows);
    if (need && (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < need)) return B2B_ERROR_INVALID_VALUE;
    int64_t seg;
    const bool split = lin_split(p, seqs, rows, &seg);
    b2bk::LinArgs a = lin_args(p, Q, K, V, O);
    a.cu = cu;
    a.log_decay = log_decay;
    a.s0 = state_in;
    a.s1 = state_out;
    a.part = (float*)workspace;
    a.rows = rows;
    a.seqs = seqs;
    a.seg = (int32_t)seg;
    const b2b::LinLaunch& L = p->dtype == B2B_DTYPE_F16 ? b2b::lin_f16() : b2b::lin_bf16();
    const int64_t segs = split ? rows / seg + seqs : seqs;
    a.slots = (int32_t)segs;
    if (split) {
        if (L.run(a, p->dim, true, segs, stream) != hipSuccess) return B2B_ERROR_HIP;
        if (L.scan(a, p->dim, stream) != hipSuccess) return B2B_ERROR_HIP;
    }
    return L.run(a, p->dim, false, segs, stream) == hipSuccess ? B2B_SUCCESS : B2B_ERROR_HIP;
}

b2b_status_t b2b_linear_attn_step(b2b_linear_attn_t p, int32_t batch, b2b_rows_t Q, b2b_rows_t K, b2b_rows_t V,
                                  b2b_rows_t O, const float* log_decay, const float* state_in, float* state_out,
                                  hipStream_t stream) {
    if (!p || !lin_sizes_ok(p, batch, batch)) return B2B_ERROR_INVALID_VALUE;
    if (!batch) return B2B_SUCCESS;
    if (!log_decay || !state_in || !state_out || (uintptr_t)state_in % 16 || (uintptr_t)state_out % 16)
        return B2B_ERROR_INVALID_VALUE;
    if (!lin_operands_ok(p, batch, Q, K, V, O)) return B2B_ERROR_INVALID_VALUE;
    b2bk::LinArgs a = lin_args(p, Q, K, V, O);
    a.log_decay = log_decay;
    a.s0 = state_in;
    a.s1 = state_out;
    a.rows = batch;
    const b2b::LinLaunch& L = p->dtype == B2B_DTYPE_F16 ? b2b::lin_f16() : b2b::lin_bf16();
    return L.step(a, p->dim, stream) == hipSuccess ? B2B_SUCCESS : B2B_ERROR_HIP;
}

}  // extern "C"
