// Attention as a cascade of two products: O = softmax(scale Q.K^T + mask).V,
// the scores and the probabilities kept on chip.
//
// The same rearrangement problem as in the GEMM cascades: the result of the
// first product is the second one's operand.  The first product is computed
// transposed, S^T = K.Q^T on v_mfma_f32_32x32x16 (operand: lane l holds row
// l%32 and the 8 k values 8*(l/32)+u; result: lane l holds column l%32 and
// rows 8*(r/4) + 4*(l/32) + r%4, r < 16), so a lane holds scores of one query
// row.  Its maximum and its sum over the keys are then sums over the lane's
// own registers and one exchange between the two 32-lane halves, and the
// probabilities, rounded and packed, are the second product's operand as they
// lie: O^T = V^T.P^T takes its keys in the order
//     16s + 8*(u/4) + 4*(l/32) + u%4        (K-step s, slot u)
// which V's transposing LDS reads follow.  Nothing moves between lanes, and
// O^T's accumulators again hold one query row a lane, so the softmax's
// rescaling is one factor a lane.
//
// Queries of the heads that share a key head lie side by side in a tile:
// row rr of a sequence is token rr / G, head kvh * G + rr % G.  Short
// sequences then fill tiles G times better and every key tile that is read
// serves all heads of its group.
//
// One pass over the keys with a running maximum m and sum l (log2 scale: the
// scale factor carries log2 e, and v_exp_f32 is a power of two).  m moves only
// when a row's new maximum exceeds it by more than 8: probabilities then stay
// below 2^8, which 16-bit types and fp32 sums hold as exactly as values
// below 1, and most tiles rescale nothing.  m starts at the lowest finite
// value, so that a row which sees no key needs no branch: its probabilities
// are exp2(-inf) = 0, its sum stays 0 and its output is written as 0.
#pragma once
#include "kernels_gen.hpp"

namespace b2bk {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.402823466e38f;
constexpr float kMaxLag = 8.f;     // how far (log2) a running maximum may lag behind

// Division of n < 2^31 by a number that the call fixes: with l = ceil(log2 d)
// and m = floor(2^(31+l) / d) + 1, which 32 bits hold, n / d is n m / 2^(31+l)
// rounded down.  (A prologue has half a dozen of them, 20 to 140 instructions
// each as the compiler writes them.)
struct FastDiv {
    uint32_t m;
    int32_t l, d;
    void set(int32_t by) {
        d = by;
        l = 0;
        while (((int64_t)1 << l) < d) ++l;
        m = (uint32_t)(((uint64_t)1 << (31 + l)) / (uint64_t)d + 1);
    }
    __device__ __forceinline__ int operator()(int n) const { return (int)(__umulhi(2u * (unsigned)n, m) >> l); }
};

// One operand: rows of heads, strides in elements, head_dim contiguous.
struct AttnRows {
    const void* p;
    int64_t ld, hs;     // from row to row, from head to head
};

struct AttnArgs {
    AttnRows Q, K, V;
    void* O;
    int64_t ldo, hso;
    const int32_t* cu_q;    // seqs + 1 starts (rows of Q and O); null: sequence s is row s alone
    const int32_t* cu_k;    // seqs + 1 starts (rows of K and V); null: see kv_stride
    const int32_t* lens;    // with kv_stride: keys of each sequence
    int64_t k_stride, v_stride;   // from sequence to sequence, where cu_k is null
    int64_t rows, keys;     // rows of Q; rows of K (cu_k) or the most keys of a sequence (lens)
    float* lse;             // [rows, heads], natural logarithm, or null
    float* part;            // partial results [slots, rows, heads, D], and their
    float* part_lse;        // [slots, rows, heads] log2-sum-exp2
    int32_t seqs, heads, dim, causal;
    int32_t slot0;          // the first part's slot
    FastDiv kv_heads, group, splits;    // splits: parts of the keys
    int32_t tiles;          // row tiles (the grid's bound)
    float sc;               // scale * log2 e
    // where part i of n key tiles begins (n <= 2^25, at most 64 parts; n splits as
    // whole * parts + rest, so that nothing leaves 31 bits)
    __device__ __forceinline__ int part_at(int n, int i) const {
        const int whole = splits(n), rest = n - whole * splits.d;
        return whole * i + splits(rest * i);
    }
};

// ---------------------------------------------------------------------------
// Where a workgroup works
// ---------------------------------------------------------------------------
struct SeqTile {
    int seq, local, tiles;   // sequence, tile within it, tiles it has
    int q0, nq;              // first row of Q, rows (tokens)
    int k0, nk;              // first key, keys
};

// Sequence starts come from device memory: clamped to the rows there are, so
// that no values of theirs lead outside the tensors.
__device__ __forceinline__ void seq_range(const int32_t* cu, int s, int total, int* start, int* n) {
    int a = cu[s], b = cu[s + 1];
    a = a < 0 ? 0 : (a > total ? total : a);
    b = b < a ? a : (b > total ? total : b);
    *start = a;
    *n = b - a;
}

// Sum over this lane and those below it.
__device__ __forceinline__ int lanes_sum(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);   // row_shr:1, 2, 4, 8: sums within 16 lanes
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);   // row_bcast:15 into rows 1 and 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);   // row_bcast:31 into rows 2 and 3
    return x;
}

// Largest of this lane's and those below it (not negative).
__device__ __forceinline__ int lanes_max(int x) {
    auto up = [&](int y) { x = x > y ? x : y; };
    up(__builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false));
    up(__builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false));
    up(__builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false));
    up(__builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false));
    up(__builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false));
    up(__builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false));
    return x;
}

// The sequence and place of tile `tile`, a sequence of n tokens having
// ceil(n * group / bm) tiles, and at least `least`: every wave scans the
// starts 64 at a time.  cu_k may be null.
__device__ __forceinline__ bool find_tile(const int32_t* cu_q, const int32_t* cu_k, int seqs, int rows, int keys, int group,
                                          int bm, int least, int tile, SeqTile* out) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int s0 = 0; s0 < seqs; s0 += 64) {
        const int s = s0 + lane;
        int q0 = 0, n = 0, k0 = 0, nk = 0, mine = 0;
        if (s < seqs) {
            seq_range(cu_q, s, rows, &q0, &n);
            if (cu_k) seq_range(cu_k, s, keys, &k0, &nk);
            mine = (int)(((unsigned)n * (unsigned)group + (unsigned)bm - 1) / (unsigned)bm);
            mine = mine < least ? least : mine;
        }
        const int sum = lanes_sum(mine);
        const unsigned long long hit = __ballot(before + sum > tile);
        if (hit) {
            const int at = __ffsll(hit) - 1;
            out->seq = s0 + at;
            out->tiles = __builtin_amdgcn_readlane(mine, at);
            out->local = tile - before - __builtin_amdgcn_readlane(sum, at) + out->tiles;
            out->q0 = __builtin_amdgcn_readlane(q0, at);
            out->nq = __builtin_amdgcn_readlane(n, at);
            out->k0 = __builtin_amdgcn_readlane(k0, at);
            out->nk = __builtin_amdgcn_readlane(nk, at);
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

// As find_tile where there is one sequence: nothing to look for (77 tokens of 8
// heads of 64: 6.0 us on the device with the search, 5.5 so).
__device__ __forceinline__ bool only_tile(const int32_t* cu_q, const int32_t* cu_k, int rows, int keys, int group, int bm,
                                          int tile, SeqTile* out) {
    seq_range(cu_q, 0, rows, &out->q0, &out->nq);
    seq_range(cu_k, 0, keys, &out->k0, &out->nk);
    out->seq = 0;
    out->local = tile;
    out->tiles = (int)(((unsigned)out->nq * (unsigned)group + (unsigned)bm - 1) / (unsigned)bm);
    return tile < out->tiles;
}

// As find_tile, up to 64 sequences, the tiles that see the most keys first:
// workgroups are taken in order, so the launch ends on short ones (17
// sequences of up to 800 tokens, 8 key heads: 73 us in the sequences' order,
// 66 in this; 24 of up to 644 without a mask, 16 heads: 40 and 35).  A tile's level is about how many tiles' worth of tokens its
// last row sees.  Causal: one level a tile, the last tile of a sequence on
// top; else all tiles of a sequence share one.  The level is found bit by bit
// from how many tiles lie at or above one.
__device__ __forceinline__ bool find_tile_by_size(const int32_t* cu_q, const int32_t* cu_k, int seqs, int rows, int keys,
                                                  int group, int bm, bool causal, int tile, SeqTile* out) {
    const int lane = threadIdx.x & 63;
    int q0 = 0, n = 0, k0 = 0, nk = 0;
    if (lane < seqs) {
        seq_range(cu_q, lane, rows, &q0, &n);
        seq_range(cu_k, lane, keys, &k0, &nk);
    }
    const int tiles = (int)(((unsigned)n * (unsigned)group + (unsigned)bm - 1) / (unsigned)bm);
    // 1 .. 2^24: the level of the sequence's last (causal) or every tile
    int64_t seen = nk / 32 + 1;
    if (causal) {
        seen = (int64_t)nk * group / bm + 1;
        seen = seen < tiles ? tiles : seen;
    }
    const int top = tiles ? (seen > (1 << 24) ? 1 << 24 : (int)seen) : 0, whole = causal ? tiles : 1;
    auto above = [&](int level) __attribute__((always_inline)) {      // this lane's tiles at `level` and above
        const int c = top - level + 1;
        return c <= 0 ? 0 : (c >= whole ? tiles : c);
    };
    int level = 0;
    for (int bit = 1 << (31 - __clz(__builtin_amdgcn_readlane(lanes_max(top), 63) | 1)); bit; bit >>= 1)
        if (__builtin_amdgcn_readlane(lanes_sum(above(level | bit)), 63) > tile) level |= bit;
    if (!level) return false;       // not even all tiles are that many
    // tiles of this lane on that level, and the place among them
    const int higher = above(level + 1), mine = above(level) - higher, upto = lanes_sum(mine);
    const int place = tile - __builtin_amdgcn_readlane(lanes_sum(higher), 63);
    const int at = __ffsll(__ballot(upto > place)) - 1;
    out->seq = at;
    out->tiles = __builtin_amdgcn_readlane(tiles, at);
    // counted from the sequence's last tile
    out->local = __builtin_amdgcn_readlane(higher - upto + mine, at) + place;
    out->q0 = __builtin_amdgcn_readlane(q0, at);
    out->nq = __builtin_amdgcn_readlane(n, at);
    out->k0 = __builtin_amdgcn_readlane(k0, at);
    out->nk = __builtin_amdgcn_readlane(nk, at);
    return true;
}

// ---------------------------------------------------------------------------
// Pieces shared by the kernels
// ---------------------------------------------------------------------------
__device__ __forceinline__ float other_half(float x) {
    unsigned a = __builtin_bit_cast(unsigned, x), b = a;
    swap32(a, b);      // a: low half's value in the high lanes; b: high half's in the low ones
    const unsigned l = threadIdx.x & 32;
    return __builtin_bit_cast(float, l ? a : b);
}

// One of the two values in a word.
template <int DT>
__device__ __forceinline__ float attn_unpack(unsigned w, int hi) {
    if constexpr (DT == DT_BF16) {
        const unsigned x = hi ? (w & 0xFFFF0000u) : (w << 16);
        return __builtin_bit_cast(float, x);
    } else {
        const h2_t v = __builtin_bit_cast(h2_t, w);
        return hi ? (float)v[1] : (float)v[0];
    }
}

// Query rows as the first product's operand: lane l holds row l%32, columns
// 16s + 8*(l/32) + u; columns past D read as zero.
template <int KS>
__device__ __forceinline__ void attn_load_q(u4_t (&q)[KS], const AttnArgs& a, int64_t q0, int kvh, int rr, int rows,
                                            int lane) {
    const int h = lane >> 5;
    const int pos = a.group(rr), g = rr - pos * a.group.d;
    const char* p = (const char*)a.Q.p + ((q0 + pos) * a.Q.ld + (int64_t)(kvh * a.group.d + g) * a.Q.hs + 8 * h) * 2;
#pragma unroll
    for (int s = 0; s < KS; ++s) q[s] = u4_t{0, 0, 0, 0};
    if (rr >= rows) return;
    if (a.dim == 16 * KS) {
#pragma unroll
        for (int s = 0; s < KS; ++s) q[s] = *(const u4_t*)(p + 32 * s);
    } else {
#pragma unroll
        for (int s = 0; s < KS; ++s)
            if (16 * s + 8 * h < a.dim) q[s] = *(const u4_t*)(p + 32 * s);
    }
}

// LDS form of a tile of key or value rows: blocks of 32 columns, `R` rows x 64
// bytes each.  Keys' 16-byte chunks are XORed with bits 2-3 of the row, so the
// 16 rows that one pass of a 16-byte fragment read covers fall on all banks
// once; values stay in order, and a transposing read's 4 rows are 256
// consecutive bytes.
// Copies row group rg (16 rows) of every block; one instruction moves
// 16 rows x 64 bytes.  Rows past the resource and columns past D read as zero.
template <int DB, int R, bool SWZ>
__device__ __forceinline__ void attn_copy(const unsigned char* dst, __amdgpu_buffer_rsrc_t rs, int ld2, int dim, int rg,
                                          int lane) {
    const int row = 16 * rg + (lane >> 2);
    const int chunk = SWZ ? ((lane & 3) ^ ((row >> 2) & 3)) : (lane & 3);
    const int off = row * ld2 + chunk * 16;
#pragma unroll
    for (int b = 0; b < DB; ++b)
        lds_dma16<false>(rs, dst + b * R * 64 + rg * 1024, 32 * b + 8 * chunk < dim ? off + 64 * b : -16);
}

// resource of key rows [row, row + n) of one head
__device__ __forceinline__ __amdgpu_buffer_rsrc_t attn_rsrc(const void* p, int64_t row, int64_t ld, int64_t at, int n,
                                                            int dim) {
    return make_rsrc((const char*)p + (row * ld + at) * 2, n > 0 ? (uint32_t)(((n - 1) * ld + dim) * 2) : 0u);
}

template <int DT>
__device__ __forceinline__ u4_t attn_pack(const f16x_t& s, int k) {
    return u4_t{Ty<DT>::pack(s[8 * k], s[8 * k + 1]), Ty<DT>::pack(s[8 * k + 2], s[8 * k + 3]),
                Ty<DT>::pack(s[8 * k + 4], s[8 * k + 5]), Ty<DT>::pack(s[8 * k + 6], s[8 * k + 7])};
}

// A value fragment: 32 columns of block `t`, K-step `ks` (16 rows), in the
// relabelled key order; vb: the lane's base.
template <int R>
__device__ __forceinline__ u4_t attn_vfrag(const unsigned char* v, int vb, int t, int ks) {
    u4_t out;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        auto* p = (__attribute__((address_space(3))) unsigned char*)(lds_ptr_t)v + vb + t * R * 64 + 1024 * ks + 512 * e;
        const u2_t w = __builtin_bit_cast(
            u2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) tr4_t*)p));
        out[2 * e] = w[0];
        out[2 * e + 1] = w[1];
    }
    return out;
}
__device__ __forceinline__ int attn_vbase(int lane) {
    const int g = lane >> 4, i = lane & 15;
    return (4 * (g >> 1) + (i >> 2)) * 64 + 32 * (g & 1) + 8 * (i & 3);
}
// A key fragment's address for even (0) and odd (1) K-steps.
__device__ __forceinline__ int attn_kbase(int lane, int odd) {
    const int row = lane & 31, c = 2 * odd + (lane >> 5);
    return row * 64 + ((c ^ ((row >> 2) & 3)) << 4);
}

// Whether any sequence holds this lane's row, which 16 lanes share; every lane
// of the wave is active.  from, to: where lane's sequence of the first 64 starts
// and ends, which the caller has asked for early.  (Starts may be in any order,
// so it takes a look at each sequence.)
__device__ __forceinline__ bool in_a_sequence(const AttnArgs& a, int row, int from, int to) {
    const int lane = threadIdx.x & 63;
    bool in = false;
    for (int s0 = 0;;) {
        // (a row is 0 .. rows - 1, so clamping changes nothing here)
        const bool have = s0 + lane < a.seqs;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int r = __builtin_amdgcn_readlane(row, 16 * g);
            in |= __ballot(have && r >= from && r < to) && lane >> 4 == g;
        }
        s0 += 64;
        if (s0 >= a.seqs || __all(in)) return in;
        const int s = s0 + lane < a.seqs ? s0 + lane : a.seqs - 1;
        from = a.cu_q[s];
        to = a.cu_q[s + 1];
    }
}

// The softmax state of one query row a lane.
struct RowState {
    float m, l;
    __device__ __forceinline__ void init() { m = kLowest; l = 0.f; }
};

// The largest of a lane's scores (its half of the keys).
template <int NK>
__device__ __forceinline__ float attn_max(const f16x_t (&s)[NK]) {
    float mx = s[0][0];
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int r = 0; r < 16; ++r) mx = __builtin_fmaxf(mx, s[k][r]);
    return mx;
}

// Moves the running maximum (and rescales O and l) where the rows' largest
// scores ask for it.
template <int NO>
__device__ __forceinline__ void attn_move_max(float mx, RowState& st, f16x_t (&o)[NO], float sc) {
    mx = __builtin_fmaxf(mx, other_half(mx)) * sc;
    if (__any(mx - st.m > kMaxLag)) {
        const float m1 = __builtin_fmaxf(st.m, mx);
        const float alpha = __builtin_amdgcn_exp2f(st.m - m1);
        st.m = m1;
        st.l *= alpha;
#pragma unroll
        for (int t = 0; t < NO; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[t][r] *= alpha;
    }
}

// Scores -> probabilities, in place, and their sum.
template <int NK>
__device__ __forceinline__ void attn_probs(f16x_t (&s)[NK], RowState& st, float sc) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            s[k][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k][r], sc, -st.m));
            sum += s[k][r];
        }
    st.l += sum;
}

// Masks scores of keys at or past `lim` (counted from the tile's first key,
// less 4 for the upper half of the lanes).
template <int NK>
__device__ __forceinline__ void attn_mask(f16x_t (&s)[NK], int lim) {
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if (32 * k + 8 * (r >> 2) + (r & 3) >= lim) s[k][r] = -__builtin_inff();
}

// Writes one query row: the output (rounded to the type, 8 consecutive columns
// a store after a swap of lane halves), or the partial result in fp32.
template <int DT, int DB, bool PART>
__device__ __forceinline__ void attn_store(const AttnArgs& a, const f16x_t (&o)[DB], const RowState& st, int64_t q0,
                                           int kvh, int rr, int rows, int slot, int lane) {
    const int h = lane >> 5;
    const float l = st.l + other_half(st.l);
    // l: a NaN (from a NaN among the row's scores) goes through to the output
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int pos = a.group(rr), head = kvh * a.group.d + (rr - pos * a.group.d);
    const int64_t row = q0 + pos;
    const bool live = rr < rows;
    const float lse2 = l == 0.f ? -__builtin_inff() : st.m + __builtin_amdgcn_logf(l);
    // `FULL`: no columns past D
    auto columns = [&](auto FULL) __attribute__((always_inline)) {
        if constexpr (PART) {
            const int64_t at = ((int64_t)slot * a.rows + row) * a.heads + head;
            if (!live) return;
            if (h == 0) a.part_lse[at] = lse2;
#pragma unroll
            for (int t = 0; t < DB; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int c = 32 * t + 8 * q + 4 * h;
                    if (FULL.value || c < a.dim)
                        *(f4_t*)(a.part + at * a.dim + c) = f4_t{o[t][4 * q] * inv, o[t][4 * q + 1] * inv,
                                                                 o[t][4 * q + 2] * inv, o[t][4 * q + 3] * inv};
                }
        } else {
            if (live && h == 0 && a.lse) a.lse[row * a.heads + head] = lse2 * kLn2;
            char* p = (char*)a.O + (row * a.ldo + (int64_t)head * a.hso) * 2;
            u4_t w[2 * DB];
#pragma unroll
            for (int t = 0; t < DB; ++t)
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    unsigned x0 = Ty<DT>::pack(o[t][4 * q] * inv, o[t][4 * q + 1] * inv);
                    unsigned x1 = Ty<DT>::pack(o[t][4 * q + 2] * inv, o[t][4 * q + 3] * inv);
                    unsigned y0 = Ty<DT>::pack(o[t][4 * q + 4] * inv, o[t][4 * q + 5] * inv);
                    unsigned y1 = Ty<DT>::pack(o[t][4 * q + 6] * inv, o[t][4 * q + 7] * inv);
                    swap32(x0, y0);
                    swap32(x1, y1);
                    w[2 * t + q / 2] = u4_t{x0, x1, y0, y1};
                }
            if (!live) return;
#pragma unroll
            for (int i = 0; i < 2 * DB; ++i)
                if (FULL.value || 16 * i + 8 * h < a.dim) *(u4_t*)(p + 2 * (16 * i + 8 * h)) = w[i];
        }
    };
    if (a.dim == 32 * DB) columns(std::true_type{});
    else columns(std::false_type{});
}

// Infinities and NaN among the values, causal.  A tile of the second product
// multiplies the probability 0 of an unseen key by that key's value, which
// gives NaN where the value is not finite.  So a wave whose results are not all
// finite (looked at once, behind the last tile) computes its rows again, by
// itself and straight from memory, values that are not finite left out; for each
// column it remembers the first key that had one, of each kind, and gives it to
// the rows that see that key.  Where every row is computed again 4096 causal rows
// of 32 heads of 128 take 2.2 ms instead of 0.15.  (A row with a NaN among its
// scores is NaN throughout and needs none of it.)
template <class C>
__device__ __forceinline__ bool attn_finite(const f16x_t (&o)[C::DB], const RowState& st) {
    float z = 0.f;
#pragma unroll
    for (int b = 0; b < C::DB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) z = __builtin_fmaf(o[b][r], 0.f, z);
    const unsigned long long odd = __ballot(z != 0.f), nan = __ballot(st.l != st.l);
    return !((unsigned)(odd | odd >> 32) & ~(unsigned)(nan | nan >> 32));
}

// Tiles [t0, t1) of a sequence's nk keys from row k0 on; lim: as for attn_mask.
// Few registers before speed: those that the tiles' loop has must do.
template <class C>
__device__ __forceinline__ void attn_again(const AttnArgs& a, f16x_t (&o)[C::DB], const RowState& st, int64_t q0, int64_t k0,
                                           int nk, int kvh, int rr, int rows, int lim, int t0, int t1, int lane) {
    using M = Ty32<C::DT>;
    constexpr unsigned kExp = C::DT == DT_BF16 ? 0x7F80 : 0x7C00;
    const int m = lane & 31, h = lane >> 5;
    const int pos = a.group(rr), head = kvh * a.group.d + (rr - pos * a.group.d);
    const char* q = (const char*)a.Q.p + ((q0 + pos) * a.Q.ld + (int64_t)head * a.Q.hs + 8 * h) * 2;
    int first[3][C::DB];          // of +inf, -inf and NaN in column 32b + m
#pragma unroll
    for (int b = 0; b < C::DB; ++b) {
        o[b] = f16x_t{};
        first[0][b] = first[1][b] = first[2][b] = 0x7FFFFFFF;
    }
    for (int t = t0; t < t1; ++t) {
        f16x_t s[1] = {f16x_t{}};
        const int key = t * C::BN + m;
        const char* k = (const char*)a.K.p + ((k0 + key) * a.K.ld + kvh * a.K.hs + 8 * h) * 2;
#pragma unroll 1
        for (int j = 0; j < C::KS; ++j) {
            const bool in = 16 * j + 8 * h < a.dim;
            u4_t x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
            if (in && key < nk) x = *(const u4_t*)(k + 32 * j);
            if (in && rr < rows) y = *(const u4_t*)(q + 32 * j);
            s[0] = M::mma(x, y, s[0]);
        }
        attn_mask<1>(s, lim - t * C::BN);
#pragma unroll
        for (int r = 0; r < 16; ++r) s[0][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[0][r], a.sc, -st.m));
#pragma unroll
        for (int b = 0; b < C::DB; ++b)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                u4_t x = {0, 0, 0, 0};
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int at = t * C::BN + 16 * ks + 8 * (u >> 2) + 4 * h + (u & 3), c = 32 * b + m;
                    unsigned v = 0;
                    if (at < nk && c < a.dim)
                        v = *(const unsigned short*)((const char*)a.V.p + ((k0 + at) * a.V.ld + kvh * a.V.hs + c) * 2);
                    if ((v & kExp) == kExp) {
                        const int kind = v & 0x7FFF & ~kExp ? 2 : (int)(v >> 15);
#pragma unroll
                        for (int i = 0; i < 3; ++i)
                            if (i == kind && at < first[i][b]) first[i][b] = at;
                        v = 0;
                    }
                    x[u >> 1] |= v << (16 * (u & 1));
                }
                o[b] = M::mma(x, attn_pack<C::DT>(s[0], ks), o[b]);
                __builtin_amdgcn_sched_barrier(0);
            }
    }
    const int seen = lim + 4 * h;
    const float give[3] = {__builtin_inff(), -__builtin_inff(), __builtin_nanf("")};
#pragma unroll
    for (int b = 0; b < C::DB; ++b)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int other = __shfl_xor(first[i][b], 32), all = first[i][b] < other ? first[i][b] : other;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int c = 8 * (r >> 2) + (r & 3);
                const int x0 = __builtin_amdgcn_readlane(all, c), x1 = __builtin_amdgcn_readlane(all, c + 4);
                if (seen > (h ? x1 : x0)) o[b][r] += give[i];
            }
        }
}

// ---------------------------------------------------------------------------
// Many rows: a workgroup's waves take 32 rows each and share the key tiles
// ---------------------------------------------------------------------------
// Tiles of 32 keys, two slots of LDS, a wave's queries in registers: 168
// registers and 32 KB at D = 128, which leaves room for three workgroups a
// compute unit.  One's matrix instructions run under the others' softmax (a
// tile of 32 x 32 scores: 512 cycles of matrix instructions, some 350 of vector
// ones, at D = 128).  Two workgroups with tiles of 64 keys and the next tile's
// scores computed ahead did as well on one long sequence and lost on short ones
// (8001 packed tokens: 77 us, 72 so), whose time is a workgroup's start: its
// place found, first keys and queries waited for (some 12 of its 38 thousand
// cycles).
// A third slot of LDS, keys asked for two tiles ahead, was slower (packed tokens
// 65.6 us -> 67.1, 16384 tokens 2015 -> 2023).
// Measured: 16384 causal tokens, 32 heads of 128 (8 key heads), bf16: 1.94 to 2.0
// ms by the card, 1105 to 1143 TFLOP/s of the 1154 to 1228 that a product of 8192^3
// reaches there (matrix cores busy 0.66 of the cycles, the clock held down by
// power); 8001 tokens in 17 sequences: 66 to 68 us; head dim 64, half of the matrix
// work for the same softmax: 9000 tokens of 16 heads in 24 sequences 34 to 35 us
// (500 to 520 TFLOP/s), bound by the longest sequences' chains of tiles at the
// launch's end (compute units busy 0.70) and, while busy, by vector instructions.
template <int DT_, int DB_, bool PART_>
struct AttnCfg {
    static constexpr int DT = DT_, DB = DB_, WAVES = 4, THREADS = 64 * WAVES;
    static constexpr bool PART = PART_;
    static constexpr int BM = 32 * WAVES, BN = 32;
    static constexpr int KS = 2 * DB;                       // K-steps of the first product
    static constexpr int TILE = BN * DB * 64, LDS_BYTES = 4 * TILE;
    static_assert(LDS_BYTES <= 160 * 1024, "LDS");
};

template <class C>
__device__ __forceinline__ void attn_tile_body(const AttnArgs& a, unsigned char* lds, int block) {
    using M = Ty32<C::DT>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int rest = a.kv_heads(block), kvh = block - rest * a.kv_heads.d;
    const int tile = C::PART ? a.splits(rest) : rest, split = rest - tile * a.splits.d;
    SeqTile w;
    if (a.cu_q) {
        const bool found = a.seqs == 1 ? only_tile(a.cu_q, a.cu_k, (int)a.rows, (int)a.keys, a.group.d, C::BM, tile, &w)
                           : a.seqs <= 64 ? find_tile_by_size(a.cu_q, a.cu_k, a.seqs, (int)a.rows, (int)a.keys, a.group.d, C::BM,
                                                            a.causal, tile, &w)
                                        : find_tile(a.cu_q, a.cu_k, a.seqs, (int)a.rows, (int)a.keys, a.group.d, C::BM, 0,
                                                    tile, &w);
        if (!found) return;
    } else {
        // all rows are one sequence's
        w.q0 = w.k0 = 0;
        w.nq = (int)a.rows;
        w.nk = (int)a.keys;
        w.tiles = a.tiles;
        w.local = tile;
    }
    const int64_t k0 = w.k0;
    const int nk = w.nk;
    // the last tile of a causal sequence sees the most keys: it starts first
    const int row0 = (a.causal ? w.tiles - 1 - w.local : w.local) * C::BM;
    const int rows = w.nq * a.group.d, shift = nk - w.nq;
    auto sees = [&](int rr) -> int {     // keys that row rr sees
        if (rr >= rows) return 0;
        if (!a.causal) return nk;
        const int n = a.group(rr) + 1 + shift;
        return n < 0 ? 0 : n;
    };
    const int last = (row0 + C::BM < rows ? row0 + C::BM : rows) - 1;
    const int end = sees(last);                               // keys the workgroup needs
    const int nt = (end + C::BN - 1) / C::BN;
    const int t0 = C::PART ? a.part_at(nt, split) : 0, t1 = C::PART ? a.part_at(nt, split + 1) : nt;
    const int wrow = row0 + 32 * wave;                        // this wave's first row
    const int rr = wrow + (lane & 31);
    const int lim = sees(rr) - 4 * (lane >> 5);
    u4_t q[C::KS];
    f16x_t o[C::DB];
    RowState st;
    st.init();
#pragma unroll
    for (int t = 0; t < C::DB; ++t) o[t] = f16x_t{};
    // tiles below `clear` need no mask (they are full and every row of the wave sees them)
    const int clear = wrow + 32 <= rows ? sees(wrow) / C::BN : 0;
    // tiles from `done` on show this wave nothing
    const int wlast = (wrow + 32 < rows ? wrow + 32 : rows) - 1;
    const int done = wrow < rows ? (sees(wlast) + C::BN - 1) / C::BN : 0;
    // Slots 0 and 1 hold even and odd tiles, keys then values; two waves copy
    // the keys, two the values.
    const bool keys = wave < 2;
    const AttnRows& src = keys ? a.K : a.V;
    const int64_t head_at = (int64_t)kvh * src.hs;
    auto copy = [&](int t) __attribute__((always_inline)) {
        const int n = nk - t * C::BN < C::BN ? nk - t * C::BN : C::BN;
        const unsigned char* dst = lds + (2 * (t & 1) + (keys ? 0 : 1)) * C::TILE;
        const auto rs = attn_rsrc(src.p, k0 + (int64_t)t * C::BN, src.ld, head_at, n, a.dim);
        if (keys) attn_copy<C::DB, C::BN, true>(dst, rs, (int)src.ld * 2, a.dim, wave, lane);
        else attn_copy<C::DB, C::BN, false>(dst, rs, (int)src.ld * 2, a.dim, wave - 2, lane);
    };
    const int kb0 = attn_kbase(lane, 0), kb1 = attn_kbase(lane, 1), vb = attn_vbase(lane);
    if (t0 < t1) copy(t0);
    attn_load_q<C::KS>(q, a, w.q0, kvh, rr, rows, lane);
    for (int t = t0; t < t1; ++t) {
        barrier_vm<0>();          // tile t is in LDS, and everyone is done with tile t - 1
        // the queries are taken here, where the compiler's own wait for them
        // costs nothing: behind the next copies it would wait for those too
        if (t == t0)
#pragma unroll
            for (int j = 0; j < C::KS; ++j) asm volatile("" : "+v"(q[j]));
        if (t + 1 < t1) copy(t + 1);
        if (t >= done) continue;
        const unsigned char* kt = lds + 2 * (t & 1) * C::TILE;
        const unsigned char* vt = kt + C::TILE;
        f16x_t s[1] = {f16x_t{}};
#pragma unroll
        for (int j = 0; j < C::KS; ++j)
            s[0] = M::mma(*(const u4_t*)(kt + ((j & 1) ? kb1 : kb0) + (j >> 1) * C::BN * 64), q[j], s[0]);
        if (t >= clear) attn_mask<1>(s, lim - t * C::BN);
        attn_move_max<C::DB>(attn_max<1>(s), st, o, a.sc);
        attn_probs<1>(s, st, a.sc);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const u4_t p = attn_pack<C::DT>(s[0], k);
#pragma unroll
            for (int b = 0; b < C::DB; ++b) o[b] = M::mma(attn_vfrag<C::BN>(vt, vb, b, k), p, o[b]);
        }
    }
    if (a.causal && !attn_finite<C>(o, st))
        attn_again<C>(a, o, st, w.q0, k0, nk, kvh, rr, rows, lim, t0, done < t1 ? done : t1, lane);
    attn_store<C::DT, C::DB, C::PART>(a, o, st, w.q0, kvh, rr, rows, a.slot0 + split, lane);
}

template <class C>
__global__ __launch_bounds__(C::THREADS, 3) void attn_tile_kernel(AttnArgs a) {
    __shared__ __attribute__((aligned(1024))) unsigned char lds[C::LDS_BYTES];
    attn_tile_body<C>(a, lds, blockIdx.x);
}

// ---------------------------------------------------------------------------
// Few rows (up to 32 a workgroup): the waves take different keys
// ---------------------------------------------------------------------------
// What bounds it is the bytes of K and V.  Each wave streams tiles of 32 keys
// of its own through its own LDS, without a barrier until the end.  Keys and
// values take the same 32 rows of LDS in turn (values are asked for once the
// scores are computed, the next keys once the products are), which leaves
// room for three workgroups a compute unit; their waves cover each other's
// waits.  The four waves' results are joined in LDS.
template <int DT_, int DB_>
struct AttnRowsCfg {
    static constexpr int DT = DT_, DB = DB_, WAVES = 4, THREADS = 64 * WAVES, BN = 32, KS = 2 * DB;
    static constexpr int TILE = BN * DB * 64, JOIN = WAVES * TILE;
    static constexpr int LDS_BYTES = JOIN + 2 * WAVES * 32 * 4;
    static_assert(WAVES == 4, "the join: a quarter of the columns' sums at a time");
};

template <class C>
__device__ __forceinline__ void attn_rows_body(const AttnArgs& a, unsigned char* lds, int block) {
    using M = Ty32<C::DT>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int rest = a.kv_heads(block), kvh = block - rest * a.kv_heads.d;
    const int row_tile = a.splits(rest), split = rest - row_tile * a.splits.d;
    const int seq = row_tile / a.tiles, tile = row_tile - seq * a.tiles;    // tiles: row tiles of a sequence
    const int rows = a.group.d, rr = 32 * tile + (lane & 31);
    int nk = a.lens[seq];
    nk = nk < 0 ? 0 : (nk > (int)a.keys ? (int)a.keys : nk);
    nk = __builtin_amdgcn_readfirstlane(nk);
    const int nt = (nk + C::BN - 1) / C::BN;
    const int t0 = a.part_at(nt, split), t1 = a.part_at(nt, split + 1);
    u4_t q[C::KS];
    f16x_t o[C::DB];
    RowState st;
    attn_load_q<C::KS>(q, a, seq, kvh, rr, rows, lane);
    st.init();
#pragma unroll
    for (int t = 0; t < C::DB; ++t) o[t] = f16x_t{};
    unsigned char* mine = lds + wave * C::TILE;
    const int64_t khead = (int64_t)kvh * a.K.hs + seq * a.k_stride, vhead = (int64_t)kvh * a.V.hs + seq * a.v_stride;
    auto copy = [&](const AttnRows& x, int64_t at, int t, auto SWZ) __attribute__((always_inline)) {
        const int n = nk - t * C::BN < C::BN ? nk - t * C::BN : C::BN;
        const auto rs = attn_rsrc(x.p, (int64_t)t * C::BN, x.ld, at, n, a.dim);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");    // what the rows held has been read
#pragma unroll
        for (int rg = 0; rg < 2; ++rg) attn_copy<C::DB, C::BN, SWZ.value>(mine, rs, (int)x.ld * 2, a.dim, rg, lane);
    };
    const int kb0 = attn_kbase(lane, 0), kb1 = attn_kbase(lane, 1), vb = attn_vbase(lane);
    if (t0 + wave < t1) copy(a.K, khead, t0 + wave, std::true_type{});
    for (int t = t0 + wave; t < t1; t += C::WAVES) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        f16x_t s[1] = {f16x_t{}};
#pragma unroll
        for (int j = 0; j < C::KS; ++j)
            s[0] = M::mma(*(const u4_t*)(mine + ((j & 1) ? kb1 : kb0) + (j >> 1) * C::BN * 64), q[j], s[0]);
        copy(a.V, vhead, t, std::false_type{});
        if ((t + 1) * C::BN > nk) attn_mask<1>(s, nk - t * C::BN - 4 * (lane >> 5));
        attn_move_max<C::DB>(attn_max<1>(s), st, o, a.sc);
        attn_probs<1>(s, st, a.sc);
        u4_t p[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) p[k] = attn_pack<C::DT>(s[0], k);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int b = 0; b < C::DB; ++b)
#pragma unroll
            for (int k = 0; k < 2; ++k) o[b] = M::mma(attn_vfrag<C::BN>(mine, vb, b, k), p[k], o[b]);
        if (t + C::WAVES < t1) copy(a.K, khead, t + C::WAVES, std::true_type{});
    }
    // join: every wave's maximum and sum, then its rows, scaled to the common maximum
    float* ms = (float*)(lds + C::JOIN);           // [maximum, sum][wave][row]
    const float l = st.l + other_half(st.l);
    if (lane < 32) {
        ms[wave * 32 + lane] = st.m;
        ms[(C::WAVES + wave) * 32 + lane] = l;
    }
    __syncthreads();
    float m = kLowest, sum = 0.f;
#pragma unroll
    for (int v = 0; v < C::WAVES; ++v) m = __builtin_fmaxf(m, ms[v * 32 + (lane & 31)]);
#pragma unroll
    for (int v = 0; v < C::WAVES; ++v)
        sum += ms[(C::WAVES + v) * 32 + (lane & 31)] * __builtin_amdgcn_exp2f(ms[v * 32 + (lane & 31)] - m);
    const float f = __builtin_amdgcn_exp2f(st.m - m) * (sum == 0.f ? 0.f : 1.f / sum);
    const int64_t at0 = ((int64_t)(a.slot0 + split) * a.rows + seq) * a.heads + kvh * a.group.d;
    if (wave == 0 && lane < 32 && rr < rows)
        a.part_lse[at0 + rr] = sum == 0.f ? -__builtin_inff() : m + __builtin_amdgcn_logf(sum);
    const int live = rows - 32 * tile < 32 ? rows - 32 * tile : 32;
    // half of the columns at a time: a wave's tile of LDS holds 32 rows of
    // 16 DB floats, [column quad][row]
    float* mo = (float*)mine;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        __syncthreads();
#pragma unroll
        for (int x = 0; x < 2 * C::DB; ++x) {
            const int y = half * 2 * C::DB + x, b = y / 4, g = y % 4;        // column quads 2y and 2y + 1
            *(f4_t*)(mo + ((2 * x + (lane >> 5)) * 32 + (lane & 31)) * 4) =
                f4_t{o[b][4 * g] * f, o[b][4 * g + 1] * f, o[b][4 * g + 2] * f, o[b][4 * g + 3] * f};
        }
        __syncthreads();
        for (int i = threadIdx.x; i < live * 4 * C::DB; i += C::THREADS) {
            const int row = i / (4 * C::DB), c = i % (4 * C::DB), col = 4 * (half * 4 * C::DB + c);
            if (col >= a.dim) continue;
            f4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < C::WAVES; ++x) {
                const f4_t y = *(const f4_t*)((const float*)(lds + x * C::TILE) + (c * 32 + row) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += y[e];
            }
            *(f4_t*)(a.part + (at0 + 32 * tile + row) * a.dim + col) = v;
        }
    }
}

// One launch for both kinds of keys of a batch behind a shared prefix: its
// first workgroups take the prefix (bound by the matrix cores), the others
// the requests' own keys (bound by memory); they fit a compute unit together.
// 128 requests behind 32768 tokens, up to 1000 own keys, 32 heads of 128: 124 us
// on the device (the products alone 58, the bytes alone 77: a prefix tile a
// wave takes about 1.1 us however few its neighbours are, so the two hide each
// other in part only; own workgroups spread among the prefix's: 137 at best).
// 32 behind 4097, up to 512 own: 15.3 us and 4.5 for the join.
template <int DT, int DB>
__global__ __launch_bounds__(256, 3) void attn_prefix_kernel(AttnArgs p, AttnArgs own, int prefix_blocks) {
    using C = AttnCfg<DT, DB, true>;
    using R = AttnRowsCfg<DT, DB>;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[C::LDS_BYTES > R::LDS_BYTES ? C::LDS_BYTES : R::LDS_BYTES];
    if ((int)blockIdx.x < prefix_blocks) attn_tile_body<C>(p, lds, blockIdx.x);
    else attn_rows_body<R>(own, lds, blockIdx.x - prefix_blocks);
}

// ---------------------------------------------------------------------------
// Joining partial results: 16 lanes a (row, head), 8 columns a lane
// ---------------------------------------------------------------------------
// O = sum_s w_s O_s / sum_s w_s with w_s = 2^(lse_s - max); parts that saw no
// key have lse = -inf and weight 0.  One pass with a running maximum, three or
// four parts' loads in flight.  SUB = 4: the quarters of a wave take every fourth
// part of one (row, head) each, for few rows of many parts, whose time is the
// loads' latency (32 rows of 32 heads in 17 parts: 6.0 us by 16 lanes, 4.6 so);
// else it is the parts' bytes (2500 rows of 24 heads of 96 in two parts, 47 MB
// read: 10.7 us).
// A row that belongs to no sequence has no partial results, and its output stays
// as it is.
template <int DT, int SUB>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int slots) {
    constexpr int PER = SUB == 1 ? 3 : 4;       // parts' loads in flight
    const int lane = threadIdx.x & 15, sub = SUB == 1 ? 0 : (threadIdx.x >> 4) & (SUB - 1);
    // (rows x heads stays below 2^31)
    const int n = (int)a.rows * a.heads, mine = (int)blockIdx.x * (16 / SUB) + (int)threadIdx.x / (16 * SUB);
    // places past the last stay, as copies of it that write nothing: every lane looks at sequences
    const int at = mine < n ? mine : n - 1, row = at / a.heads;
    int from = 0, to = 0;
    if (a.cu_q) {
        const int s = (int)(threadIdx.x & 63) < a.seqs ? threadIdx.x & 63 : a.seqs - 1;
        from = a.cu_q[s];
        to = a.cu_q[s + 1];
    }
    const int head = at - row * a.heads;
    float m = -__builtin_inff(), sum = 0.f, x[8] = {};
    const bool live = 8 * lane < a.dim;
    const float* p = a.part + (int64_t)at * a.dim + 8 * lane;
    const int64_t slot = (int64_t)n * a.dim;
    float least = __builtin_inff();     // of the parts that saw keys
    // to a new maximum (0 for -inf: nothing has been seen)
    auto scale_to = [&](float m1) __attribute__((always_inline)) {
        const float f = __builtin_amdgcn_exp2f(m - m1);
        sum *= f;
        // a weight of 0 leaves its part out, whatever that holds
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = f == 0.f ? 0.f : x[e] * f;
    };
    for (int s0 = sub; s0 < slots; s0 += PER * SUB) {
        float w[PER], m1 = m;
        f4_t v[PER][2];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool in = s0 + i * SUB < slots;
            const int s = in ? s0 + i * SUB : s0;
            w[i] = in ? a.part_lse[(int64_t)s * n + at] : -__builtin_inff();
            v[i][0] = v[i][1] = f4_t{0.f, 0.f, 0.f, 0.f};
            if (live) {
                v[i][0] = *(const f4_t*)(p + s * slot);
                v[i][1] = *(const f4_t*)(p + s * slot + 4);
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) m1 = __builtin_fmaxf(m1, w[i]);
        const float m0 = m1 == -__builtin_inff() ? 0.f : m1;
        scale_to(m0);
        m = m1;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float f = __builtin_amdgcn_exp2f(w[i] - m0);
            sum += f;
            least = __builtin_fminf(least, w[i] == -__builtin_inff() ? __builtin_inff() : w[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = f == 0.f ? x[e] : __builtin_fmaf(f, v[i][e >> 2][e & 3], x[e]);
        }
    }
    if constexpr (SUB > 1) {
        float m1 = m;
#pragma unroll
        for (int d = 16; d < 16 * SUB; d <<= 1) m1 = __builtin_fmaxf(m1, __shfl_xor(m1, d));
        scale_to(m1 == -__builtin_inff() ? 0.f : m1);
        m = m1;
#pragma unroll
        for (int d = 16; d < 16 * SUB; d <<= 1) {
            sum += __shfl_xor(sum, d);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += __shfl_xor(x[e], d);
        }
    }
    if (__any(least - m < -126.f)) {
        // a part's weight may have been 0: its infinities and NaN are not left out
#pragma unroll 1
        for (int s = 0; s < slots; ++s)
            if (live && a.part_lse[(int64_t)s * n + at] != -__builtin_inff())
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float y = p[s * slot + e];
                    if (!(__builtin_fabsf(y) <= -kLowest)) x[e] += y;
                }
    }
    if ((a.cu_q && !in_a_sequence(a, row, from, to)) || mine >= n || sub) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (live)
        *(u4_t*)((char*)a.O + ((int64_t)row * a.ldo + (int64_t)head * a.hso + 8 * lane) * 2) =
            u4_t{Ty<DT>::pack(x[0] * inv, x[1] * inv), Ty<DT>::pack(x[2] * inv, x[3] * inv),
                 Ty<DT>::pack(x[4] * inv, x[5] * inv), Ty<DT>::pack(x[6] * inv, x[7] * inv)};
    if (lane == 0 && a.lse) a.lse[at] = sum == 0.f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(sum)) * kLn2;
}

}  // namespace b2bk
