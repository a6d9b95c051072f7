// C ABI of attention under a window and over pages (b2b_attn.h): checks, how a
// call is laid over workgroups, launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attn_plan.hpp"
#include "paged_attn_launch.hpp"

namespace {

using namespace b2b;

// Workgroups that a call's key tiles are cut for: two a compute unit (2048 rows of 4
// sequences behind up to 16384 keys, 32 heads of 128, with the join: 362 us, 378 at
// 768, 376 at 1024), and four times as many of sequences of few rows (64 requests of
// up to 8192 keys: 221 us at 512, 204 at 1024, 201 at 2048).
constexpr int kTarget = 512;
// Key tiles of a part, at least: below 512 keys a second launch takes longer than
// the four waves of one workgroup do (3 requests of up to 300 keys: 10.5 us cut, 7.1 whole).
constexpr int kLeast = 16;

// Under a window, with as many row tiles as workgroups are wanted, nothing is cut
// while the keys before a sequence's rows make no row tile longer than this, or than
// the others take together (a row tile's start and end cost some 7 key tiles, 256 run
// at full rate: n of them take n / 36 key tiles' time at least).  Cutting costs the
// join's launch where row tiles are alike and a multiple where they are not (520 row
// tiles, 32 heads of 128 on 8 key heads: all behind a window of 512, 22 key tiles,
// 38 us whole and 42 cut; 1000: 58 and 62; 4096: 196 and 201; one chunk of 64 rows
// behind as much, 60 prompts of 40 behind nothing: 22 and 27, 32 and 30, 88 and 34,
// behind 100000 keys 2240 and 166).
constexpr int kFar = 32;

struct Layout {
    int64_t tiles;          // row tiles a key head, at most
    int64_t items;          // workgroups a key head, at most
    int64_t granules;       // of partial results, a key head, at most (0: nothing is cut)
    int64_t subs;           // granules of a row tile
    size_t bytes;
};

// keys: the most that a sequence may have; before: the most that come before its rows
Layout lay_out(const b2b_attn_plan* p, int64_t seqs, int64_t rows, int64_t keys, int64_t before) {
    const int64_t group = p->heads / p->kv_heads;
    Layout l = {};
    l.tiles = rows * group / b2bk::kKeyRows + seqs;
    // key tiles of a row tile, at most
    int64_t most = ceil_div(keys, 32), far = ceil_div(before, 32);
    if (p->window) {
        const int64_t w = ((int64_t)p->window + b2bk::kKeyRows) / 32 + ceil_div(p->sinks, 32) + 2;
        most = std::min(most, w);
        far = std::min(far, w);
    }
    const int64_t wgs = rows * group / b2bk::kKeyRows * p->kv_heads;
    const bool enough = p->window && wgs >= kTarget && far <= std::max<int64_t>(kFar, wgs / 32);
    l.items = l.tiles;
    l.subs = rows * group <= 32 ? 1 : b2bk::kKeyRows / 32;
    if (most > kLeast && !enough) {
        l.items += 4 * kTarget / p->kv_heads;
        l.granules = std::min<int64_t>(l.subs * l.items, 8 * kTarget / p->kv_heads);
    }
    l.bytes = (size_t)l.granules * p->kv_heads * 32 * (p->dim + 1) * 4;
    return l;
}

bool key_sizes_ok(const b2b_attn_plan* p, int64_t seqs, int64_t rows, int64_t keys) {
    // (rows and keys of 2^30 at most keep every place less a window in 32 bits)
    return sizes_ok(p, seqs, rows, keys) && rows <= INT32_MAX / 2;
}

bool ready(const Layout& l, const b2b_attn_plan* p, const void* workspace, size_t bytes) {
    if (l.bytes && (!workspace || (uintptr_t)workspace % 16 || bytes < l.bytes)) return false;
    return std::max(l.items + 8, l.subs * l.tiles) * p->kv_heads <= INT32_MAX;
}

b2b_status_t launch_keys(b2b_attn_t p, const Layout& l, b2bk::KeyArgs& a, int where, void* workspace, hipStream_t stream) {
    a.causal = 1;
    a.window = (int32_t)std::min<int64_t>(p->window, std::max<int64_t>(a.keys, 1));     // (0 stays 0)
    a.sinks = (int32_t)std::min<int64_t>(p->sinks, a.keys);
    a.split = l.granules > 0;
    a.least = kLeast;
    a.per = (float)p->kv_heads / kTarget;
    a.granules = (int32_t)l.granules;
    a.subs = !a.cu_q && a.group.d <= 32 ? 1 : (int32_t)l.subs;
    a.part = (float*)workspace;
    a.part_lse = a.part + (size_t)l.granules * p->kv_heads * 32 * p->dim;
    // Few rows a sequence, on average: the few rows' kernel, heads over all XCDs (see
    // key_attn_kernel).  32 heads of 128 on 8, against the other kernel: 128 single tokens
    // behind up to 8000 keys under a window of 1024 120 us and 125, 64 behind up to 4000
    // 113 and 115, 512 behind up to 512 127 and 122.  A chunk among them goes along, 1000
    // rows with 200 single tokens behind up to 4000: that begins its prompt 374 and 385,
    // behind 8192 keys 457 and 418, of which a window leaves 1024 220 and 211.
    a.spread = a.rows * a.group.d <= (int64_t)32 * a.seqs;
    const int64_t items = a.spread ? ceil_div(l.items, 8) * 8 : l.items;
    const KeyLaunch& L = p->dtype == B2B_DTYPE_F16 ? key_attn_f16() : key_attn_bf16();
    if (L.run(a, where, (unsigned)(items * p->kv_heads), stream) != hipSuccess) return B2B_ERROR_HIP;
    if (a.split && L.join(a, where, (unsigned)(a.subs * l.tiles * p->kv_heads), stream) != hipSuccess) return B2B_ERROR_HIP;
    return B2B_SUCCESS;
}

b2bk::KeyArgs key_args(const b2b_attn_plan* p, int32_t seqs, int64_t rows, int64_t keys, const b2b_rows_t& Q,
                       const b2b_rows_t& O, const int32_t* cu_q, float* lse) {
    b2bk::KeyArgs a = {};
    base_args(p, a);
    a.Q = dev(Q, p->dim);
    a.O = const_cast<void*>(O.data);
    a.ldo = O.row_stride;
    a.hso = O.head_stride;
    a.cu_q = cu_q;
    a.rows = rows;
    a.keys = keys;
    a.lse = lse;
    a.seqs = seqs;
    return a;
}

}  // namespace

b2b_status_t b2b::window_workspace(b2b_attn_t p, int32_t seqs, int64_t rows, int64_t keys, size_t* bytes) {
    if (!key_sizes_ok(p, seqs, rows, keys)) return B2B_ERROR_INVALID_VALUE;
    *bytes = seqs && rows ? lay_out(p, seqs, rows, keys, std::max<int64_t>(keys - rows, 0)).bytes : 0;
    return B2B_SUCCESS;
}

b2b_status_t b2b::window_run(b2b_attn_t p, int32_t seqs, int64_t rows, int64_t keys, const b2b_rows_t& Q, const b2b_rows_t& K,
                             const b2b_rows_t& V, const b2b_rows_t& O, const int32_t* cu_q, const int32_t* cu_k, float* lse,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!key_sizes_ok(p, seqs, rows, keys)) return B2B_ERROR_INVALID_VALUE;
    const Extent o = extent(O, rows, p->heads, p->dim);
    if (!apart(o, {extent(Q, rows, p->heads, p->dim)}) ||
        (keys && !apart(o, {extent(K, keys, p->kv_heads, p->dim), extent(V, keys, p->kv_heads, p->dim)})))
        return B2B_ERROR_INVALID_VALUE;
    const Layout l = lay_out(p, seqs, rows, keys, std::max<int64_t>(keys - rows, 0));
    if (!ready(l, p, workspace, workspace_bytes)) return B2B_ERROR_INVALID_VALUE;
    b2bk::KeyArgs a = key_args(p, seqs, rows, keys, Q, O, cu_q, lse);
    a.K = b2b::dev(K, p->dim);
    a.V = b2b::dev(V, p->dim);
    a.cu_k = cu_k;
    return launch_keys(p, l, a, b2bk::KEYS_PACKED, workspace, stream);
}

extern "C" {

b2b_status_t b2b_attn_create_window(b2b_attn_t* plan, b2b_dtype_t dtype, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                    float scale, int32_t window, int32_t sinks) {
    if (!plan) return B2B_ERROR_INVALID_VALUE;
    *plan = nullptr;
    if (window < 1 || window > 1 << 30 || sinks < 0 || sinks > 1 << 30) return B2B_ERROR_INVALID_VALUE;
    return create_attn(plan, dtype, heads, kv_heads, head_dim, scale, true, window, sinks, 0);
}

b2b_status_t b2b_paged_attn_create(b2b_attn_t* plan, b2b_dtype_t dtype, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                   int32_t page_size, float scale, int32_t window, int32_t sinks) {
    if (!plan) return B2B_ERROR_INVALID_VALUE;
    *plan = nullptr;
    if (page_size < 1 || page_size > 1 << 20 || window < 0 || window > 1 << 30 || sinks < 0 || sinks > 1 << 30 ||
        (sinks && !window))
        return B2B_ERROR_INVALID_VALUE;
    return create_attn(plan, dtype, heads, kv_heads, head_dim, scale, true, window, sinks, page_size);
}

b2b_status_t b2b_paged_attn_workspace(b2b_attn_t p, int32_t seqs, int64_t rows, int32_t width, size_t* bytes) {
    if (!p || !bytes || !p->page || width < 0 || !key_sizes_ok(p, seqs, rows, (int64_t)width * p->page))
        return B2B_ERROR_INVALID_VALUE;
    *bytes = seqs && rows ? lay_out(p, seqs, rows, (int64_t)width * p->page, (int64_t)width * p->page).bytes : 0;
    return B2B_SUCCESS;
}

b2b_status_t b2b_paged_attn_run(b2b_attn_t p, int32_t seqs, int64_t rows, b2b_rows_t Q, b2b_pages_t K, b2b_pages_t V,
                                int32_t pages, const int32_t* table, int32_t width, int64_t table_stride, const int32_t* lens,
                                const int32_t* cu_q, b2b_rows_t O, float* lse, void* workspace, size_t workspace_bytes,
                                hipStream_t stream) {
    if (!p || !p->page || width < 0 || pages < 0) return B2B_ERROR_INVALID_VALUE;
    const int64_t keys = pages ? (int64_t)width * p->page : 0;
    if (!key_sizes_ok(p, seqs, rows, (int64_t)width * p->page) || (!cu_q && rows != seqs)) return B2B_ERROR_INVALID_VALUE;
    if (!seqs || !rows) return B2B_SUCCESS;
    if (!rows_ok(Q, rows, p->dim) || !out_ok(O, rows, p->heads, p->dim) || (uintptr_t)lse % 4) return B2B_ERROR_INVALID_VALUE;
    if (!lens) return B2B_ERROR_INVALID_VALUE;
    if (keys && (!pages_ok(K, pages) || !pages_ok(V, pages) || !table || table_stride < 0 || table_stride > kMaxFar ||
                 (seqs > 1 && table_stride < width)))
        return B2B_ERROR_INVALID_VALUE;
    const Extent o = extent(O, rows, p->heads, p->dim);
    if (!apart(o, {extent(Q, rows, p->heads, p->dim)}) ||
        (keys && !apart(o, {extent(K, pages, p->page, p->kv_heads, p->dim), extent(V, pages, p->page, p->kv_heads, p->dim)})))
        return B2B_ERROR_INVALID_VALUE;
    // (by the table's width alone, as the _workspace call)
    const Layout l = lay_out(p, seqs, rows, (int64_t)width * p->page, (int64_t)width * p->page);
    if (!ready(l, p, workspace, workspace_bytes)) return B2B_ERROR_INVALID_VALUE;
    b2bk::KeyArgs a = key_args(p, seqs, rows, keys, Q, O, cu_q, lse);
    a.pk = dev(K);
    a.pv = dev(V);
    a.table = table;
    a.table_ld = table_stride;
    a.page.set(p->page);
    a.pages = pages;
    a.lens = lens;
    // pages of whole groups of 16 rows, whose addresses the kernel works out in 32 bits
    auto near = [&](const b2b_pages_t& x) {
        return x.row_stride <= kMaxStride && x.row_stride * p->page <= INT32_MAX && x.page_stride <= INT32_MAX;
    };
    const bool whole = p->page % 16 == 0 && near(K) && near(V);
    return launch_keys(p, l, a, whole ? b2bk::KEYS_PAGES16 : b2bk::KEYS_PAGES, workspace, stream);
}

}  // extern "C"
