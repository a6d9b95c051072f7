// Attention plans and what the C entries of all attention operators check alike.
#pragma once
#include <climits>
#include <cstdint>

#include <algorithm>

#include "attn_launch.hpp"
#include "b2b_attn.h"
#include "extent.hpp"
#include "paged_attn.hpp"

struct b2b_attn_plan {
    int dtype, heads, kv_heads, dim;
    float scale;
    bool causal;
    int window, sinks;      // window 0: every earlier key
    int page;               // keys a page; 0: contiguous keys
};

namespace b2b {

constexpr int64_t kMaxStride = (int64_t)1 << 23;    // 64 rows' offsets stay below 2^30 bytes
constexpr int64_t kMaxFar = (int64_t)1 << 40;       // from head to head, request to request: past any memory

// Rows of heads that the kernels can address: n rows, 16-byte pieces.
inline bool rows_ok(const b2b_rows_t& r, int64_t n, int dim) {
    if (!r.data || (uintptr_t)r.data % 16) return false;
    if (r.row_stride % 8 || r.head_stride % 8 || r.head_stride < 0 || r.head_stride > kMaxFar) return false;
    return n <= 1 || (r.row_stride >= dim && r.row_stride <= kMaxStride);
}
// Rows that are written: no two of their (row, head) share an element.
inline bool out_ok(const b2b_rows_t& r, int64_t n, int heads, int dim) {
    if (!rows_ok(r, n, dim) || (heads > 1 && r.head_stride < dim)) return false;
    return n <= 1 || heads <= 1 || r.row_stride >= (heads - 1) * r.head_stride + dim ||
           r.head_stride >= (n - 1) * r.row_stride + dim;
}
inline b2bk::AttnRows dev(const b2b_rows_t& r, int dim) {
    // a single row's stride is never stepped by; the kernels still size resources with it
    return {r.data, r.row_stride >= dim && r.row_stride <= kMaxStride ? r.row_stride : dim, r.head_stride};
}

// Pages that the kernels can address, 16-byte pieces.
inline bool pages_ok(const b2b_pages_t& x, int64_t pages) {
    if (!x.data || (uintptr_t)x.data % 16) return false;
    for (int64_t s : {x.page_stride, x.row_stride, x.head_stride})
        if (s % 8 || s < 0 || s > kMaxFar) return false;
    return x.page_stride <= ((int64_t)1 << 46) / std::max<int64_t>(pages, 1);
}
inline Extent extent(const b2b_rows_t& r, int64_t n, int heads, int dim) {
    return Extent(r.data, dim, {{n, r.row_stride}, {heads, r.head_stride}});
}
inline Extent extent(const b2b_pages_t& x, int64_t pages, int64_t size, int heads, int dim) {
    return Extent(x.data, dim, {{pages, x.page_stride}, {size, x.row_stride}, {heads, x.head_stride}});
}
// Whether what is written shares no element with any of the others.
inline bool apart(const Extent& o, std::initializer_list<Extent> others) {
    for (const Extent& x : others)
        if (overlap(o, x)) return false;
    return true;
}
inline b2bk::Pages dev(const b2b_pages_t& x) { return {x.data, x.page_stride, x.row_stride, x.head_stride}; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool sizes_ok(const b2b_attn_plan* p, int64_t seqs, int64_t rows, int64_t keys) {
    return seqs >= 0 && rows >= 0 && keys >= 0 && rows <= INT32_MAX && rows * (int64_t)p->heads <= INT32_MAX - 1024 &&
           keys <= INT32_MAX / 2 && seqs <= INT32_MAX / 2;
}

template <class Args>
inline void base_args(const b2b_attn_plan* p, Args& a) {
    a.heads = p->heads;
    a.kv_heads.set(p->kv_heads);
    a.group.set(p->heads / p->kv_heads);
    a.dim = p->dim;
    a.sc = p->scale * b2bk::kLog2e;
    a.splits.set(1);
}

// b2b_attn_create and those for a window or pages, which check what they add
b2b_status_t create_attn(b2b_attn_t* plan, b2b_dtype_t dtype, int32_t heads, int32_t kv_heads, int32_t head_dim, float scale,
                         bool causal, int32_t window, int32_t sinks, int32_t page);

// Runs of plans with a window (contiguous keys).
b2b_status_t window_workspace(b2b_attn_t p, int32_t seqs, int64_t rows, int64_t keys, size_t* bytes);
b2b_status_t window_run(b2b_attn_t p, int32_t seqs, int64_t rows, int64_t keys, const b2b_rows_t& Q, const b2b_rows_t& K,
                        const b2b_rows_t& V, const b2b_rows_t& O, const int32_t* cu_q, const int32_t* cu_k, float* lse,
                        void* workspace, size_t workspace_bytes, hipStream_t stream);

}  // namespace b2b
