// Norms of queries and keys for each head and their rotation, in one pass over
// the heads; for new tokens, keys and values into the pages of a cache.
//
//   y = x / sqrt(mean(x^2) + eps) * weight,   pair (a, b) of y -> (a cos t - b sin t, b cos t + a sin t)
//
// What bounds it is the bytes: every head is read once and written once.  L
// lanes hold a head, 8 elements each (L = 8 up to 64 elements, 16 up to 128): one
// 16-byte load and store a lane, the sum of squares by exchanges inside L lanes.
// The partner of element i is rotary_dim / 2 away, a whole number of 4-element
// halves of a lane's piece, which lanes fetch from each other.
//
// A row's angles are the same for all of its heads: a workgroup of R rows works
// out R x rotary_dim / 2 sines and cosines once, in LDS, and a lane keeps those of
// its 8 elements in registers over the heads it takes.  An angle is position x
// frequency / 2 pi in float64, of which only the fraction of a turn counts: off by
// 2^-24 of a turn at positions of 2^31 and frequencies up to 1.
//
// Measured (bf16, 32 + 8 heads of 128, normed): 8001 rows, 164 MB, in 34 us on the
// device (a copy of as many bytes 32.6), 32768 rows in 125 us, 5.4 TB/s.  Few rows
// take the latencies one after another: positions, angles, heads, 3.7 us for 3 rows;
// appended, starts and lengths before them, 5.4 us for 128 rows and 11.4 for 4097 of
// 16 + 4 + 4 heads of 64 (5 by their bytes).
#pragma once
#include "paged_attn.hpp"

namespace b2bk {

constexpr int kRotaryRows = 8;

struct RotaryArgs {
    AttnRows Q, K, V;               // V: append only
    void *Qo, *Ko;
    int64_t ldqo, hqo, ldko, hko;
    Pages ck, cv;                   // append: where keys and values go
    const int32_t *table, *lens, *cu;
    int64_t table_ld;
    const int32_t* positions;       // [axes, rows]; null: a row's place in its sequence
    int64_t position_ld;
    const void *qw, *kw;
    double turns[64];               // frequency / 2 pi of each pair
    uint8_t axis[64];
    FastDiv page, per_row;          // per_row: workgroups that share R rows' heads
    int32_t rows, seqs, pages, width, heads, kv_heads, dim, rotary, axes, row_log;    // R = 1 << row_log, up to kRotaryRows
    float eps;
};

// Sum over the L lanes (8 or 16) that hold a head, in each of them.
template <int L>
__device__ __forceinline__ float head_sum(float x) {
    auto add = [&](int y) { x += __builtin_bit_cast(float, y); };
    auto me = [&] { return __builtin_bit_cast(int, x); };
    add(__builtin_amdgcn_update_dpp(0, me(), 0xB1, 0xf, 0xf, false));       // lane ^ 1
    add(__builtin_amdgcn_update_dpp(0, me(), 0x4E, 0xf, 0xf, false));       // lane ^ 2
    add(__builtin_amdgcn_update_dpp(0, me(), 0x141, 0xf, 0xf, false));      // 7 - lane of 8
    if constexpr (L == 16) add(__builtin_amdgcn_update_dpp(0, me(), 0x140, 0xf, 0xf, false));   // 15 - lane of 16
    return x;
}
template <int L>
__device__ __forceinline__ double head_sum(double x) {
#pragma unroll
    for (int d = 1; d < L; d <<= 1) x += __shfl_xor(x, d);
    return x;
}

template <int DT>
__device__ __forceinline__ void unpack8(u4_t w, float (&x)[8]) {
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = attn_unpack<DT>(w[u >> 1], u & 1);
}

// A head's 8 elements a lane: out = inv (x own + partner's x far), where `own` and
// `far` are cosine and signed sine with the weights of either element folded in.
// Elements meet them before the norm's factor: in float32 while the head's sum of
// squares is below `most`, 2^126 (elements below 2^63), or for no sum where a weight
// lies outside 2^-60 to 2^60 (bf16 alone has such weights).
struct Turn {
    float own[8], far[8], most;
};

// Whether any lane of the wave holds a bf16 weight outside 2^-60 to 2^60, 0 apart (two at a time, as integers).
__device__ __forceinline__ bool far_weights(u4_t w) {
    typedef unsigned short us2_t __attribute__((ext_vector_type(2)));
    us2_t big = {0, 0}, small = {0xFFFF, 0xFFFF};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const us2_t m = __builtin_bit_cast(us2_t, w[i] & 0x7FFF7FFFu);
        big = __builtin_elementwise_max(big, m);
        small = __builtin_elementwise_min(small, (us2_t)(m - (unsigned short)1));      // (0 becomes the largest)
    }
    return __any(big[0] > 0x5D80 || big[1] > 0x5D80 || small[0] < 0x217F || small[1] < 0x217F);
}

// APPEND: keys and values go to the pages.  NORM, INTER: the plan's flags.
template <int DT, int L, bool APPEND, bool NORM, bool INTER>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a) {
    // Heads in flight a lane.  Two, for more workgroups a compute unit, but where the
    // norm's steps a head leave the loads more to cover and nothing is appended (8001
    // rows of 40 heads of 128: 38.0 us with 2, 36.1 with 4, 38.6 with 8; without a norm,
    // 5003 rows of 28 heads of 96: 14.4, 15.3, 16.1; 4097 rows into pages: 12.0, 12.6, 12.7).
    constexpr int GROUPS = 256 / L, BATCH = L == 16 && NORM && !APPEND ? 4 : 2;
    constexpr int ROWS = kRotaryRows, TURNS = ROWS / 4;      // angles a thread works out, at most
    __shared__ float turn[ROWS][64][2];             // [row][pair][cos, sin]
    // append: a row's place in its sequence, or kNoRow of none, and the page that holds it (-1: none)
    constexpr int kNoRow = -0x7FFFFFFF - 1;
    __shared__ int place[ROWS], row_page[ROWS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int R = 1 << a.row_log, block = a.per_row((int)blockIdx.x), share = (int)blockIdx.x - block * a.per_row.d;
    const int row0 = block << a.row_log;
    const int group = threadIdx.x / L, c = threadIdx.x & (L - 1);
    const int r = group & (R - 1), row = row0 + r;
    // this lane's heads: Q's, then K's, then V's, `step` apart
    const int step = (GROUPS >> a.row_log) * a.per_row.d, first = (group >> a.row_log) + share * (GROUPS >> a.row_log);
    const int keys0 = a.heads, values0 = a.heads + a.kv_heads, items = values0 + (APPEND ? a.kv_heads : 0);
    const bool live = row < a.rows && 8 * c < a.dim;
    // the next heads from item i0 on, below `end`, of an operand whose first head is item i1
    auto fetch = [&](auto& raw, const AttnRows& x, int i1, int i0, int end) __attribute__((always_inline)) {
        const char* p = (const char*)x.p + (row * x.ld + (int64_t)(i0 - i1) * x.hs + 8 * c) * 2;
#pragma unroll
        for (int j = 0; j < (int)(sizeof(raw) / 16); ++j) {
            raw[j] = u4_t{0, 0, 0, 0};
            if (live && i0 + j * step < end) raw[j] = *(const u4_t*)(p + j * step * x.hs * 2);
        }
    };
    // what a lane starts with is asked for at once: keys and values wait behind the same latency
    const int first_k = keys0 > first ? first + (keys0 - first + step - 1) / step * step : first;
    const int first_v = values0 > first ? first + (values0 - first + step - 1) / step * step : first;
    u4_t rq[BATCH], rk[2], rv[2];
    fetch(rq, a.Q, 0, first, keys0);
    fetch(rk, a.K, keys0, first_k, values0);
    if constexpr (APPEND) fetch(rv, a.V, values0, first_v, items);
    // the partners of this lane's elements
    const int half = a.rotary >> 1;
    int from[2];                // lane (of L) with the partner of each half of the piece
    const int other = (half >> 2) & 1;      // whether it is in the other half of that lane's piece
    bool turned[2], lower[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int v = 2 * c + h;            // 4-element unit
        turned[h] = 4 * v < a.rotary;
        lower[h] = 4 * v < half;
        from[h] = turned[h] ? (lower[h] ? v + (half >> 2) : v - (half >> 2)) >> 1 : c;
    }
    auto partner = [&](u4_t w) __attribute__((always_inline)) {
        u4_t out;
        if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < 4; ++i) out[i] = w[i] >> 16 | w[i] << 16;
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 2; ++j) out[2 * h + j] = __shfl(other ? w[2 * (h ^ 1) + j] : w[2 * h + j], from[h], L);
        }
        return out;
    };
    u4_t qw = {0, 0, 0, 0}, kw = qw;
    if constexpr (NORM) {
        if (a.qw && 8 * c < a.dim) qw = *((const u4_t*)a.qw + c);
        if (a.kw && 8 * c < a.dim) kw = *((const u4_t*)a.kw + c);
    }
    // pair threadIdx.x / R (and 256 / R on) of row threadIdx.x % R: its frequency and position
    double turns[TURNS];
    int at[TURNS];
#pragma unroll
    for (int t = 0; t < TURNS; ++t) {
        const int i = threadIdx.x + 256 * t, p = i >> a.row_log, mine = row0 + (i & (R - 1));
        turns[t] = 0.0;
        at[t] = 0;
        if (p < half && mine < a.rows) {
            turns[t] = a.turns[p];
            if (!APPEND || a.positions) at[t] = a.positions[(a.axes > 1 ? a.axis[p] * a.position_ld : 0) + mine];
        }
    }
    [[maybe_unused]] int page_entry[ROWS / 4];
    if constexpr (APPEND) {
        // a wave takes every fourth row: which sequence holds it, and its page, which is looked up under the sines
        int seq[ROWS / 4], spot[ROWS / 4];
#pragma unroll
        for (int x = 0; x < ROWS / 4; ++x) {
            const int rr = wave + 4 * x, mine = row0 + rr;
            seq[x] = -1;
            spot[x] = 0;
            if (!a.cu && rr < R && mine < a.rows) {
                seq[x] = mine;
                spot[x] = (a.lens[mine] > 0 ? a.lens[mine] : 0) - 1;
            }
        }
        if (a.cu)
            for (int s0 = 0; s0 < a.seqs; s0 += 64) {
                const int s = s0 + lane;
                int q0 = 0, n = 0, len = 0;
                if (s < a.seqs) {
                    seq_range(a.cu, s, a.rows, &q0, &n);
                    len = a.lens[s] > 0 ? a.lens[s] : 0;
                }
                bool all = true;
#pragma unroll
                for (int x = 0; x < ROWS / 4; ++x) {
                    const int rr = wave + 4 * x, mine = row0 + rr;
                    if (rr >= R || seq[x] >= 0) continue;
                    const unsigned long long hit = __ballot(mine >= q0 && mine < q0 + n);
                    if (hit) {
                        const int l = __ffsll(hit) - 1;
                        seq[x] = s0 + l;
                        spot[x] = __builtin_amdgcn_readlane(len, l) -
                                  (__builtin_amdgcn_readlane(q0, l) + __builtin_amdgcn_readlane(n, l) - mine);
                    } else {
                        all = false;
                    }
                }
                if (all) break;
            }
#pragma unroll
        for (int x = 0; x < ROWS / 4; ++x) {
            const int rr = wave + 4 * x;
            page_entry[x] = -1;
            if (rr >= R) continue;
            if (lane == 0) place[rr] = seq[x] < 0 ? kNoRow : spot[x];
            const int pg = spot[x] >= 0 ? a.page(spot[x]) : 0;
            if (seq[x] >= 0 && spot[x] >= 0 && pg < a.width) page_entry[x] = a.table[seq[x] * a.table_ld + pg];
        }
        __syncthreads();
    }
#pragma unroll
    for (int t = 0; t < TURNS; ++t) {
        const int i = threadIdx.x + 256 * t, p = i >> a.row_log, rr = i & (R - 1);
        if (p >= half) break;
        if (APPEND && !a.positions) at[t] = row0 + rr < a.rows ? place[rr] : 0;
        const double x = at[t] * turns[t];
        float s, co;
        sincospif(2.f * (float)(x - __builtin_rint(x)), &s, &co);
        turn[rr][p][0] = co;
        turn[rr][p][1] = s;
    }
    if constexpr (APPEND)
#pragma unroll
        for (int x = 0; x < ROWS / 4; ++x)
            if (wave + 4 * x < R && lane == 0) row_page[wave + 4 * x] = page_entry[x];
    __syncthreads();
    auto turn_of = [&](const void* weight, u4_t w) __attribute__((always_inline)) {
        Turn t;
        float x[8], y[8];
        if (NORM && weight) {
            unpack8<DT>(w, x);
            unpack8<DT>(partner(w), y);
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = y[u] = 1.f;
        }
        t.most = 0x1p126f;
        if constexpr (NORM && DT == DT_BF16)
            if (far_weights(w)) t.most = 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int e = 8 * c + u;
            const int p = (INTER ? e >> 1 : (lower[u >> 2] ? e : e - half)) & 63;
            const float co = turned[u >> 2] ? turn[r][p][0] : 1.f, s = turned[u >> 2] ? turn[r][p][1] : 0.f;
            t.own[u] = x[u] * co;
            t.far[u] = (INTER ? !(u & 1) : lower[u >> 2]) ? -s * y[u] : s * y[u];
        }
        return t;
    };
    char *kp = nullptr, *vp = nullptr;      // append: where head 0's piece of the row goes
    bool writes = live;
    if constexpr (APPEND) {
        const int spot = writes ? place[r] : kNoRow, entry = writes ? row_page[r] : -1;
        writes = spot != kNoRow;            // (a row of no sequence writes nothing)
        if (entry >= 0 && entry < a.pages) {
            const int in = spot - a.page(spot) * a.page.d;
            kp = (char*)a.ck.p + (entry * a.ck.ps + in * a.ck.ld + 8 * c) * 2;
            vp = (char*)a.cv.p + (entry * a.cv.ps + in * a.cv.ld + 8 * c) * 2;
        }
    } else {
        kp = (char*)a.Ko + (row * a.ldko + 8 * c) * 2;
    }
    const bool all = a.rotary == a.dim;
    const float per = 1.f / a.dim;
    auto head = [&](u4_t w, const Turn& t) __attribute__((always_inline)) {
        float x[8], y[8];
        unpack8<DT>(w, x);
        unpack8<DT>(partner(w), y);
        if (!all)       // an element that is not turned keeps its value whatever its neighbour holds
#pragma unroll
            for (int u = 0; u < 8; ++u) y[u] = turned[u >> 2] ? y[u] : 0.f;
        float inv = 1.f;
        if constexpr (NORM) {
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < 8; ++u) sum = __builtin_fmaf(x[u], x[u], sum);
            sum = head_sum<L>(sum);
            inv = __builtin_amdgcn_rsqf(__builtin_fmaf(sum, per, a.eps));
            // squares that leave float32's range (the sum infinite, or so small that terms
            // are lost), or that would with the weights
            const bool odd = !(sum < t.most && sum > 0x1p-100f) && sum == sum;
            if (__any(odd)) {
                double d = 0.0;
#pragma unroll
                for (int u = 0; u < 8; ++u) d += (double)x[u] * x[u];
                d = 1.0 / sqrt(head_sum<L>(d) / a.dim + (double)a.eps);
                if (odd) {
                    inv = 1.f;
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        x[u] = (float)(x[u] * d);
                        y[u] = (float)(y[u] * d);
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            x[u] = __builtin_fmaf(y[u], t.far[u], x[u] * t.own[u]);
            if constexpr (NORM) x[u] *= inv;
        }
        return u4_t{Ty<DT>::pack(x[0], x[1]), Ty<DT>::pack(x[2], x[3]), Ty<DT>::pack(x[4], x[5]), Ty<DT>::pack(x[6], x[7])};
    };
    // heads from item i0 to `end`, the first of them in `raw`: `p` is where the operand's head 0 goes, `hs` from head to head
    auto heads = [&](auto& raw, const AttnRows& x, int i1, int i0, int end, char* p, int64_t hs, const Turn* t)
                     __attribute__((always_inline)) {
        while (i0 < end) {
#pragma unroll
            for (int j = 0; j < (int)(sizeof(raw) / 16); ++j) {
                if (i0 >= end) break;
                const u4_t out = t ? head(raw[j], *t) : raw[j];
                if (p && writes) *(u4_t*)(p + (i0 - i1) * hs * 2) = out;
                i0 += step;
            }
            if (i0 < end) fetch(raw, x, i1, i0, end);
        }
    };
    if (first < keys0) {
        const Turn t = turn_of(a.qw, qw);
        heads(rq, a.Q, 0, first, keys0, (char*)a.Qo + (row * a.ldqo + 8 * c) * 2, a.hqo, &t);
    }
    if (first_k < values0) {
        const Turn t = turn_of(a.kw, kw);
        heads(rk, a.K, keys0, first_k, values0, kp, APPEND ? a.ck.hs : a.hko, &t);
    }
    if constexpr (APPEND) heads(rv, a.V, values0, first_v, items, vp, a.cv.hs, nullptr);
}

}  // namespace b2bk
