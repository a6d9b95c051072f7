// Linear attention with a decay for each head: no softmax, and a state
// instead of a cache,
//     S_t = lambda S_{t-1} + k_t v_t^T        (S: D x D, float32)
//     o_t = scale q_t^T S_t.
//
// Prompts go 32 tokens at a time.  With S the state before a chunk and i, j
// its tokens (0 ..),
//     o_i = scale ( lambda^(i+1) q_i^T S + sum_{j<=i} lambda^(i-j) (q_i.k_j) v_j )
//     S'  = lambda^n S + sum_j lambda^(n-1-j) k_j v_j^T
// -- three cascades whose intermediates stay on chip (the relabelled K order
// of the attention kernels):
//   * scores are computed transposed, S^T = K.Q^T, so decayed and rounded
//     they are the operand of V^T.P^T as they lie;
//   * the state's accumulators (lane: value column, registers: key columns,
//     their order set by the order in which the keys' columns are read) are,
//     rounded, the operand of S^T.Q^T as they lie;
//   * both end in O^T with one query row a lane, so the factor
//     scale lambda^(i+1) is one multiplication a register.
// A sequence's head is one workgroup walking its chunks in order, so what
// counts is the time of a chunk.  Half of the waves keep the state, half
// compute outputs, one of each on a SIMD, 32 value columns a wave: while a
// state wave takes in chunk c, an output wave answers chunk c's queries from
// the copy of the state that the state wave left in LDS a step before.  (All
// waves doing both in turn took 4.1 us for 64 tokens of a head of 128, two
// barriers and one wave a SIMD; two steps of 32 take 2.6 so.)  A state wave
// bounds the step: 24 matrix instructions (bf16) and 220 vector ones that wait
// for one another; two sets of state waves with half of the rows each were
// slower, their split values being computed twice.
// Measured: 8200 bf16 tokens in 9 sequences, 32 heads of 128: 83 to 87 us by the
// card (3.6 TB/s of its own bytes), the time of the longest sequence's steps;
// 32768 fp16 tokens of 16 heads: 194 to 200 us (segments' states 61, joined in 8,
// outputs 125; K and V are read twice, 5.11 TB/s would take 158).
//
// The state is float32 and so are its terms: lambda^(n-1-j) v_j is split into
// parts of the 16-bit type that together hold its 24 bits (bf16: three; fp16:
// two, of values scaled into its range), each a pass of matrix instructions with
// the exact k_j.  What ends in the 16-bit output alone is held in its type: the
// scores in two parts, and, as q's partner, a copy of the state, rounded once.
// fp16 holds neither over its range: a row's scores, and the copy, are scaled by
// powers of two that the float32 accumulators take out again, and so are a
// chunk's decayed values.  (The scaling of scores and values takes 2 % of the time
// of the 32768 tokens, and 4 % of that of the 8200 in fp16: 93 us, 97 so.)
#pragma once
#include "attn.hpp"

namespace b2bk {

struct LinArgs {
    AttnRows Q, K, V;
    void* O;
    int64_t ldo, hso;
    const int32_t* cu;          // seqs + 1 starts
    const float* log_decay;     // [heads]
    const float* s0;            // [seqs, heads, D, D] states before, or null (zero)
    float* s1;                  // states after, or null
    float* part;                // [tiles, heads, D, D]: a segment's own state, then the state before it
    int64_t rows;
    int32_t seqs, heads, kv_heads, group;
    int32_t seg, slots;         // tokens of a segment; the segments that `part` holds
    float scale;
};

// lambda^d, d >= 0, from its log2 (exact for d = 0 whatever lambda is)
__device__ __forceinline__ float lin_pow(float g2, int d) {
    return d <= 0 ? 1.f : __builtin_amdgcn_exp2f((float)d * g2);
}

// STATE: only the segments' own states (from zero), for the pass before the
// outputs of sequences that are split: no output waves, no queries.
// LDS: SLOTS chunks of keys, values (and queries), copied by the state waves
// SLOTS - 1 chunks ahead; two copies of the state; two chunks of outputs on
// their way out; the copies' exponents (fp16).
template <int DT_, int D_, bool STATE_>
struct LinCfg {
    static constexpr int DT = DT_, D = D_, DB = D / 32, C = 32;
    static constexpr bool STATE = STATE_;
    static constexpr int WAVES = STATE ? DB : 2 * DB, THREADS = 64 * WAVES;
    static constexpr int KS = 2 * DB, TILE = C * DB * 64, OPS = STATE ? 2 : 3, SLOTS = STATE ? 4 : 3;
    static constexpr int COPY = SLOTS * OPS * TILE, COPY_BYTES = DB * KS * 1024;      // a copy of the state
    static constexpr int OUT = COPY + (STATE ? 0 : 2 * COPY_BYTES);                   // two chunks of outputs
    static constexpr int EXPS = OUT + (STATE ? 0 : 2 * TILE), LDS_BYTES = EXPS + (STATE ? 0 : 64);
    static constexpr int PARTS = DT == DT_BF16 ? 3 : 2, PIECES = TILE / 1024 / DB;      // copies of a tile by a state wave
    static_assert(LDS_BYTES <= 160 * 1024 && (SLOTS - 2) * OPS * PIECES <= 63, "config");
};

// A transposed fragment of the swizzled key tile: 32 columns of block t,
// K-step ks of its rows; tb[e]: the lane's bases.  Of each 16 columns the
// second and third four trade places: the product's result then has, in lane
// half h and register r, column 16*(r/8) + 8h + r%8 of the block (lin_row),
// which makes eight registers of the state an operand in the natural order.
__device__ __forceinline__ void lin_tbase(int lane, int (&tb)[2]) {
    const int g = lane >> 4, i = lane & 15;
    const int q = ((i & 1) << 1) | ((i >> 1) & 1);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int chunk = (2 * (g & 1) + (q >> 1)) ^ (2 * e + (g >> 1));
        tb[e] = 512 * e + (4 * (g >> 1) + (i >> 2)) * 64 + chunk * 16 + (q & 1) * 8;
    }
}
__device__ __forceinline__ int lin_row(int r, int h) { return 16 * (r >> 3) + 8 * h + (r & 7); }
template <int R>
__device__ __forceinline__ u4_t lin_tfrag(const unsigned char* p, const int (&tb)[2], int t, int ks) {
    u4_t out;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        auto* q = (__attribute__((address_space(3))) unsigned char*)(lds_ptr_t)p + tb[e] + t * R * 64 + 1024 * ks;
        const u2_t w = __builtin_bit_cast(
            u2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) tr4_t*)q));
        out[2 * e] = w[0];
        out[2 * e + 1] = w[1];
    }
    return out;
}

// Two values as PARTS 16-bit parts each, packed: their sum holds 24 bits (fp16:
// of values that are scaled into its range).
template <int DT, int PARTS>
__device__ __forceinline__ void lin_split(float x, float y, unsigned (&out)[PARTS]) {
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        out[p] = Ty<DT>::pack(x, y);
        if (p + 1 < PARTS) {
            // The remainder is taken from the bits that the instruction gets.
            // Left alone, the compiler may round the product behind x to fp16 once
            // for those bits and twice for the remainder (seen: one value in
            // thousands, a step apart at a tie).
            asm("" : "+v"(out[p]));
            x -= attn_unpack<DT>(out[p], 0);
            y -= attn_unpack<DT>(out[p], 1);
        }
    }
}

// What rounding left of eight values of x: their second parts.
template <int DT>
__device__ __forceinline__ u4_t lin_rest(const f16x_t& x, int k, u4_t& first) {
    u4_t out;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        unsigned w = first[i];
        asm("" : "+v"(w));          // as in lin_split
        first[i] = w;
        out[i] = Ty<DT>::pack(x[8 * k + 2 * i] - attn_unpack<DT>(w, 0), x[8 * k + 2 * i + 1] - attn_unpack<DT>(w, 1));
    }
    return out;
}

// The exponent e for which the state's largest magnitude times 2^-e is about
// 2^13: fp16 copies of larger or much smaller states would leave its range.
// Uniform over the wave; 0 for states that are in range as they are; -126 or
// above, so that 2^e and 2^-e are both finite and normal (smaller states have
// few bits left, and their copy holds them all).
template <int NT>
__device__ __forceinline__ int lin_exponent(const f16x_t (&s)[NT]) {
    float m = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) m = __builtin_fmaxf(m, __builtin_fabsf(s[t][r]));
    if (!__any(m > 16384.f) && __any(m > 0.25f)) return 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = __builtin_fmaxf(m, __shfl_xor(m, d));
    if (m > 3e38f) {       // an infinity sets no scale for the others
        m = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float x = __builtin_fabsf(s[t][r]);
                m = x <= 3e38f ? __builtin_fmaxf(m, x) : m;
            }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) m = __builtin_fmaxf(m, __shfl_xor(m, d));
    }
    if (!(m > 0.f)) return 0;
    const int e = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_frexp_expf(m) - 13);
    return e < -126 ? -126 : e;
}

// The power of two that takes m (2^-100 or more) to 2^13 .. 2^14, and its
// inverse.
__device__ __forceinline__ float lin_scale(float m, float* back) {
    const unsigned e = __builtin_bit_cast(unsigned, m) & 0x7F800000u;
    *back = __builtin_bit_cast(float, e - (13u << 23));
    return __builtin_bit_cast(float, (267u << 23) - e);
}

// That of a row's scores (its two lanes hold 16 each): fp16 operands then hold
// scores of any size, to 2^-38 of the row's largest in two parts.  A largest
// below 2^-14 counts as 2^-14: scores are then held to 2^-52, and 32 times that
// times any fp16 value is below a result's smallest step.  NaN are passed over, an
// infinity stays one.  (32768 tokens of 16 heads: 188 us without, 189 so.)
__device__ __forceinline__ float lin_row_scale(const f16x_t& p, float* up) {
    float m = 0x1p-14f;
#pragma unroll
    for (int r = 0; r < 16; ++r) m = __builtin_fmaxf(m, __builtin_fabsf(p[r]));
    return lin_scale(__builtin_fmaxf(m, other_half(m)), up);
}

// Whether one of a lane's packed values is not finite.
typedef unsigned short us2_t __attribute__((ext_vector_type(2)));
template <int DT, int N>
__device__ __forceinline__ bool lin_odd(const u4_t (&x)[N]) {
    us2_t m[4] = {};
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m[i] = __builtin_elementwise_max(m[i], __builtin_bit_cast(us2_t, x[n][i] & 0x7FFF7FFFu));
    const us2_t y = __builtin_elementwise_max(__builtin_elementwise_max(m[0], m[1]), __builtin_elementwise_max(m[2], m[3]));
    constexpr unsigned short inf = DT == DT_BF16 ? 0x7F80 : 0x7C00;
    return y[0] >= inf || y[1] >= inf;
}

// acc, or NaN if one of eight packed values is not finite (0 times it).
template <int DT>
__device__ __forceinline__ float lin_watch(const u4_t& w, float acc) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if constexpr (DT == DT_BF16)
            acc = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf2_t, (unsigned)w[i]), bf2_t{}, acc, false);
        else
            acc = __builtin_amdgcn_fdot2(__builtin_bit_cast(h2_t, (unsigned)w[i]), h2_t{}, acc, false);
    return acc;
}

// Infinities and NaN.  A product of 32 tokens multiplies the 0 of a key that
// comes after a row by that key's value, and makes NaN of rows before one that
// is not finite.  The outputs are watched (8 of some 90 vector instructions a
// step); a workgroup that has seen one that is not finite leaves its states
// unwritten and returns true, and goes again with CAREFUL: there a chunk with
// such values or scores adds them row by row, each over its own keys.  (With
// that branch in the only loop a step took 5 % longer.)
template <class C, bool CAREFUL>
__device__ __forceinline__ bool lin_body(const LinArgs& a, unsigned char* lds) {
    using M = Ty32<C::DT>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int h = lane >> 5, m = lane & 31;
    const int head = blockIdx.x % a.heads, tile = blockIdx.x / a.heads, kvh = head / a.group;
    SeqTile w;
    // (a sequence without tokens counts as one empty segment: its state still passes through)
    if (!find_tile(a.cu, nullptr, a.seqs, (int)a.rows, 0, 1, a.seg, 1, tile, &w)) return false;
    const bool last = w.local + 1 == w.tiles;
    if (C::STATE && last) return false;       // nobody reads what follows the last segment
    const int64_t row0 = w.q0 + (int64_t)w.local * a.seg;
    const int n = last ? w.nq - w.local * a.seg : a.seg;
    const float g2 = a.log_decay[head] * kLog2e;
    const int chunks = (n + C::C - 1) / C::C;

    bool again = false;
    int* flag = (int*)(lds + C::EXPS) + 8;      // an output that is not finite (behind the exponents)
    if (!C::STATE && threadIdx.x == 0) *flag = 0;
    const int vb = attn_vbase(lane);
    const int part = wave % C::DB, col = 32 * part + m;        // this wave's value columns
    auto slot = [&](int c) __attribute__((always_inline)) {      // where the c-th chunk taken in lies
        return lds + __builtin_amdgcn_readfirstlane(c % C::SLOTS * C::OPS * C::TILE);
    };

    if (wave < C::DB) {
        // ---- the state ----
        // this wave's pieces of a tile: 16 rows x 64 bytes of a block
        // The i-th chunk taken in is c = i, or (STATE: the contributions of
        // chunks are summed with their decays, in any order) from the last
        // back: a head whose decay has run out of float32's range is done early,
        // and what the pass reads last, the next pass reads first.
        auto chunk_of = [&](int i) __attribute__((always_inline)) { return C::STATE ? chunks - 1 - i : i; };
        auto copy = [&](const AttnRows& x, int64_t at, int i, int op, bool swz) __attribute__((always_inline)) {
            // past the end: as many copies, of nothing
            const int c = i < chunks ? chunk_of(i) : 0, live = i < chunks;
            const int left = n - c * C::C < C::C ? n - c * C::C : C::C;
            const auto rs = attn_rsrc(x.p, row0 + (int64_t)c * C::C, x.ld, at, live ? left : 0, C::D);
#pragma unroll
            for (int j = 0; j < C::PIECES; ++j) {
                const int piece = wave * C::PIECES + j, row = 16 * (piece & 1) + (lane >> 2);
                const int chunk = swz ? (lane & 3) ^ ((row >> 2) & 3) : lane & 3;
                lds_dma16<false>(rs, slot(i) + op * C::TILE + piece * 1024,
                                 row * (int)x.ld * 2 + chunk * 16 + 64 * (piece >> 1));
            }
        };
        auto copy_chunk = [&](int i) __attribute__((always_inline)) {
            copy(a.K, (int64_t)kvh * a.K.hs, i, 0, true);
            copy(a.V, (int64_t)kvh * a.V.hs, i, 1, false);
            if constexpr (!C::STATE) copy(a.Q, (int64_t)head * a.Q.hs, i, 2, true);
        };
        if (chunks > 0)
#pragma unroll
            for (int c = 0; c < C::SLOTS - 1; ++c) copy_chunk(c);
        int tb[2];
        lin_tbase(lane, tb);
        f16x_t S[C::DB];
        auto state_at = [&](float* base, int64_t at) {
            return base + (at * a.heads + head) * C::D * C::D + col;
        };
        const float* from = nullptr;
        if constexpr (!C::STATE) {
            if (w.tiles > 1) from = state_at(a.part, tile);
            else if (a.s0) from = state_at(const_cast<float*>(a.s0), w.seq);
        }
#pragma unroll
        for (int t = 0; t < C::DB; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) S[t][r] = from ? from[(32 * t + lin_row(r, h)) * C::D] : 0.f;
        // leaves a copy for the output waves, behind their next barrier
        auto leave = [&](int c) __attribute__((always_inline)) {
            if constexpr (!C::STATE) {
                unsigned char* to = lds + C::COPY + (c & 1) * C::COPY_BYTES + part * C::KS * 1024 + lane * 16;
                if constexpr (C::DT == DT_F16) {
                    const int e = lin_exponent(S);
                    const float down = __builtin_ldexpf(1.f, -e);
                    if (lane == 0) ((float*)(lds + C::EXPS))[(c & 1) * 4 + part] = __builtin_ldexpf(1.f, e);
                    if (e != 0) {
#pragma unroll
                        for (int s = 0; s < C::KS; ++s) {
                            f16x_t x = S[s >> 1];
#pragma unroll
                            for (int r = 0; r < 16; ++r) x[r] *= down;
                            *(u4_t*)(to + s * 1024) = attn_pack<C::DT>(x, s & 1);
                        }
                        return;
                    }
                }
#pragma unroll
                for (int s = 0; s < C::KS; ++s) *(u4_t*)(to + s * 1024) = attn_pack<C::DT>(S[s >> 1], s & 1);
            }
        };
        // lambda^(n-1-j) of the chunk's tokens j = 16k + 8*(i/4) + 4h + i%4
        float fall[2][8];
        auto fall_to = [&](int left) __attribute__((always_inline)) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) fall[k][i] = lin_pow(g2, left - 1 - (16 * k + 8 * (i >> 2) + 4 * h + (i & 3)));
        };
        fall_to(C::C);
        float keep = lin_pow(g2, C::C);
        if (chunks > 0) leave(0);
        for (int c = 0; c < chunks; ++c) {
            // what lies between the chunk and the segment's end
            const float after = C::STATE ? lin_pow(g2, C::C * c) : 1.f;
            if (C::STATE && __builtin_amdgcn_readfirstlane(after == 0.f)) break;
            barrier_vm<(C::SLOTS - 2) * C::OPS * C::PIECES>();   // chunk c is in LDS, and everyone is done with chunk c - 1
            copy_chunk(c + C::SLOTS - 1);
            const unsigned char* kt = slot(c);
            if (!C::STATE && n - c * C::C < C::C) {
                fall_to(n - c * C::C);
                keep = lin_pow(g2, n - c * C::C);
            }
            u4_t v[2], f[C::DB][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                v[k] = attn_vfrag<C::C>(kt + C::TILE, vb, part, k);
#pragma unroll
                for (int t = 0; t < C::DB; ++t) f[t][k] = lin_tfrag<C::C>(kt, tb, t, k);
            }
            // K-step by K-step, so that one's matrix instructions run under the
            // other's arithmetic
            u4_t vp[2][C::PARTS];
            // bf16 has float32's range, so there a chunk's decay to the
            // segment's end goes into the split values; fp16's products are
            // decayed as a whole, and its values scaled by a power of two a
            // column (a lane): two parts then hold them to 2^-38 of the column's
            // largest and 2^-23 of themselves, whatever the decays and the tokens
            // that are masked have left of them.  (Unscaled they were held to 2^-36,
            // and what the matrix instruction adds subnormal values to, to 2^-38.)
            float by = C::STATE && C::DT == DT_BF16 ? after : 1.f, back = 1.f;
            if constexpr (C::DT == DT_F16) {
                float most = 0x1p-100f;
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        most = __builtin_fmaxf(most, __builtin_fabsf(attn_unpack<C::DT>(v[k][i >> 1], i & 1) * fall[k][i]));
                by = lin_scale(__builtin_fmaxf(most, other_half(most)), &back);
            }
            auto split = [&](int k) __attribute__((always_inline)) {
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    unsigned out[C::PARTS];
                    float w0 = fall[k][2 * d], w1 = fall[k][2 * d + 1];
                    if constexpr (C::STATE || C::DT == DT_F16) {
                        w0 *= by;
                        w1 *= by;
                    }
                    lin_split<C::DT>(attn_unpack<C::DT>(v[k][d], 0) * w0, attn_unpack<C::DT>(v[k][d], 1) * w1, out);
#pragma unroll
                    for (int p = 0; p < C::PARTS; ++p) vp[k][p][d] = out[p];
                }
            };
            if constexpr (C::DT == DT_F16) {
                f16x_t u[C::DB];
#pragma unroll
                for (int t = 0; t < C::DB; ++t) u[t] = f16x_t{};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    split(k);
#pragma unroll
                    for (int p = C::PARTS - 1; p >= 0; --p)
#pragma unroll
                        for (int t = 0; t < C::DB; ++t) u[t] = M::mma(f[t][k], vp[k][p], u[t]);
                }
                const float into = C::STATE ? back * after : back;
#pragma unroll
                for (int t = 0; t < C::DB; ++t)
#pragma unroll
                    for (int r = 0; r < 16; ++r) S[t][r] = __builtin_fmaf(u[t][r], into, C::STATE ? S[t][r] : S[t][r] * keep);
            } else if constexpr (C::STATE) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    split(k);
#pragma unroll
                    for (int p = C::PARTS - 1; p >= 0; --p)
#pragma unroll
                        for (int t = 0; t < C::DB; ++t) S[t] = M::mma(f[t][k], vp[k][p], S[t]);
                }
            } else {
                // one tile of the state after the other: its copy is rounded and left
                // under the next one's matrix instructions (3 % of the launch
                // against all tiles in step; the parts' order makes no such difference)
                split(0);
                split(1);
                unsigned char* to = lds + C::COPY + ((c + 1) & 1) * C::COPY_BYTES + part * C::KS * 1024 + lane * 16;
#pragma unroll
                for (int t = 0; t < C::DB; ++t) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) S[t][r] *= keep;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int p = C::PARTS - 1; p >= 0; --p) S[t] = M::mma(f[t][k], vp[k][p], S[t]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) *(u4_t*)(to + (2 * t + k) * 1024) = attn_pack<C::DT>(S[t], k);
                }
            }
            if constexpr (!C::STATE && C::DT == DT_F16) leave(c + 1);
        }
        if (!C::STATE && chunks > 0) {
            barrier_lds();      // the output waves' last
            again = !CAREFUL && __builtin_amdgcn_readfirstlane(*flag);
        }
        float* to = nullptr;
        if constexpr (C::STATE) to = state_at(a.part, tile);
        else if (last && a.s1) to = state_at(a.s1, w.seq);
        if (to && !again)
#pragma unroll
            for (int t = 0; t < C::DB; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) to[(32 * t + lin_row(r, h)) * C::D] = S[t][r];
    } else if constexpr (!C::STATE) {
        // ---- the outputs ----
        const int kb[2] = {attn_kbase(lane, 0), attn_kbase(lane, 1)};
        float same[16];                        // decays of the scores, 0 where the key comes later
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int j = 8 * (r >> 2) + 4 * h + (r & 3);
            same[r] = j > m ? 0.f : a.scale * lin_pow(g2, m - j);
        }
        const float into = a.scale * lin_pow(g2, m + 1);
        // Outputs leave through LDS, a step later, as whole rows: in 32-byte
        // pieces straight from the registers they took 42 of 123 us (32768 tokens of
        // 16 heads of 128 whose 402 MB of reads take 81).
        constexpr int CH = 4 * C::DB, RW = 64 / CH;               // 16-byte chunks of a row; rows of a store
        auto out_at = [&](int c, int row, int chunk) __attribute__((always_inline)) {
            return lds + C::OUT + (c & 1) * C::TILE + row * CH * 16 + ((chunk ^ (row & (CH - 1))) << 4);
        };
        auto flush = [&](int c) __attribute__((always_inline)) {
            // (nothing has gone before the first chunk: a resource of no bytes takes no stores)
            const int left = c < 0 ? 0 : (n - c * C::C < C::C ? n - c * C::C : C::C);
            const auto rs = attn_rsrc(a.O, row0 + (int64_t)c * C::C, a.ldo, (int64_t)head * a.hso, left, C::D);
#pragma unroll
            for (int i = 0; i < C::C / C::DB / RW; ++i) {
                const int row = part * (C::C / C::DB) + i * RW + lane / CH, chunk = lane % CH;
                st128(rs, row * (int)a.ldo * 2 + chunk * 16, *(const u4_t*)out_at(c, row, chunk));
            }
        };
        float odd = 0.f;
        for (int c = 0; c < chunks; ++c) {
            barrier_lds();
            flush(c - 1);
            const unsigned char* kt = slot(c);
            auto rows32 = [&](const unsigned char* p, int s) __attribute__((always_inline)) {
                return *(const u4_t*)(p + kb[s & 1] + (s >> 1) * C::C * 64);
            };
            f16x_t p, y;
            float up = 1.f;           // fp16: what p and y are to be multiplied by
            const unsigned char* sp = lds + C::COPY + (c & 1) * C::COPY_BYTES + part * C::KS * 1024 + lane * 16;
            float f = into;
            if constexpr (C::DT == DT_F16) f *= ((const float*)(lds + C::EXPS))[(c & 1) * 4 + part];
            auto firsts = [&]() __attribute__((always_inline)) {
                p = y = f16x_t{};
#pragma unroll
                for (int s = 0; s < C::KS; ++s) {
                    const u4_t q = rows32(kt + 2 * C::TILE, s);
                    p = M::mma(rows32(kt, s), q, p);
                    y = M::mma(*(const u4_t*)(sp + s * 1024), q, y);
                }
                float g = f;
#pragma unroll
                for (int r = 0; r < 16; ++r) p[r] *= same[r];
                if constexpr (C::DT == DT_F16) {
                    const float down = lin_row_scale(p, &up);
                    // finite, also for the largest states: a row whose queries are 0 gets 0
                    // (where y is not 0 the result has left fp16's range long before)
                    g = __builtin_fminf(g * down, -kLowest);
#pragma unroll
                    for (int r = 0; r < 16; ++r) p[r] *= down;
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) y[r] *= g;
            };
            firsts();
            // the chunk's values and scores
            u4_t vp[4];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                vp[s] = attn_vfrag<C::C>(kt + C::TILE, vb, part, s);
                vp[2 + s] = attn_pack<C::DT>(p, s);
            }
            // The scores in two parts of the type: rounded once, they cost a row
            // of few tokens as much precision as its output's own rounding.  (The
            // output waves wait for the state waves, two passes more or not.)
#pragma unroll
            for (int s = 0; s < 2; ++s) y = M::mma(vp[s], lin_rest<C::DT>(p, s, vp[2 + s]), y);
#pragma unroll
            for (int s = 0; s < 2; ++s) y = M::mma(vp[s], vp[2 + s], y);
            if (CAREFUL && __any(lin_odd<C::DT>(vp))) {
                firsts();
                // the scores' first parts, where this wave's outputs will lie: a lane's
                // own row, read by the two lanes that hold it
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const u4_t w = attn_pack<C::DT>(p, x >> 1);
                    *(u2_t*)(out_at(c, m, 4 * part + x) + 8 * h) = u2_t{w[2 * (x & 1)], w[2 * (x & 1) + 1]};
                }
                for (int j = 0; j <= m; ++j) {
                    const float pj = attn_unpack<C::DT>(*(const unsigned short*)(out_at(c, m, 4 * part + (j >> 3)) + 2 * (j & 7)), 0);
                    const unsigned char* v = kt + C::TILE + part * C::C * 64 + j * 64 + 8 * h;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const u2_t w = *(const u2_t*)(v + 16 * x);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            y[4 * x + e] = __builtin_fmaf(pj, attn_unpack<C::DT>(w[e >> 1], e & 1), y[4 * x + e]);
                    }
                }
            }
            if constexpr (C::DT == DT_F16)
#pragma unroll
                for (int r = 0; r < 16; ++r) y[r] *= up;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const u4_t w = attn_pack<C::DT>(y, x);
                unsigned x0 = w[0], x1 = w[1], y0 = w[2], y1 = w[3];
                swap32(x0, y0);
                swap32(x1, y1);
                *(u4_t*)out_at(c, m, 4 * part + 2 * x + h) = u4_t{x0, x1, y0, y1};
                if constexpr (!CAREFUL) odd = lin_watch<C::DT>(w, odd);
            }
        }
        if (chunks > 0) {
            if (!CAREFUL && __any(odd != 0.f) && lane == 0) *flag = 1;
            barrier_lds();
            again = !CAREFUL && __builtin_amdgcn_readfirstlane(*flag);
            flush(chunks - 1);
        }
    }
    // copies of nothing still write zeros: not into LDS that is another workgroup's by then
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    return again;
}

template <class C>
__global__ __launch_bounds__(C::THREADS, 2) void lin_kernel(LinArgs a) {
    __shared__ __attribute__((aligned(1024))) unsigned char lds[C::LDS_BYTES];
    if (!lin_body<C, false>(a, lds)) return;
    if constexpr (!C::STATE) {
        barrier_lds();
        lin_body<C, true>(a, lds);
    }
}

// Segments' own states -> the state before each segment, in place.  One
// workgroup takes 1024 elements of one sequence's and head's state.
template <int D>
__global__ __launch_bounds__(256) void lin_scan_kernel(LinArgs a) {
    constexpr int PER = D * D / 1024;
    const int piece = blockIdx.x % PER, head = blockIdx.x / PER % a.heads, seq = blockIdx.x / PER / a.heads;
    // the sequence's first segment
    const int lane = threadIdx.x & 63;
    int first = 0, tiles = 0;
    for (int s0 = 0; s0 <= seq; s0 += 64) {
        const int s = s0 + lane;
        int start, n, mine = 0;
        if (s <= seq) {
            seq_range(a.cu, s, (int)a.rows, &start, &n);
            mine = n > a.seg ? (n + a.seg - 1) / a.seg : 1;
        }
        if (s0 + 64 > seq) tiles = __builtin_amdgcn_readlane(mine, seq - s0);
        const int sum = __builtin_amdgcn_readlane(lanes_sum(s < seq ? mine : 0), 63);
        first += sum;
    }
    // (starts that go back and forth would ask for more segments than there is room for)
    if (first >= a.slots) return;
    tiles = tiles < a.slots - first ? tiles : a.slots - first;
    if (tiles < 2) return;
    const float keep = lin_pow(a.log_decay[head] * kLog2e, a.seg);
    const int64_t step = (int64_t)a.heads * D * D;
    const int64_t at = (int64_t)head * D * D + piece * 1024 + threadIdx.x * 4;
    float* p = a.part + first * step + at;
    f4_t S = {0.f, 0.f, 0.f, 0.f};
    if (a.s0) S = *(const f4_t*)(a.s0 + seq * step + at);
    // eight segments' loads in flight
    for (int i0 = 0; i0 < tiles; i0 += 8) {
        f4_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i0 + i + 1 < tiles) u[i] = *(const f4_t*)(p + i * step);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i0 + i < tiles) *(f4_t*)(p + i * step) = S;
            if (i0 + i + 1 < tiles)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[e] = __builtin_fmaf(S[e], keep, u[i][e]);
        }
        p += 8 * step;
    }
}

// One token: what bounds it is reading and writing the states.  A workgroup
// takes one request's head; a thread 4 value columns of every 8th (D = 64:
// 16th) row, all loads issued before the first use.
template <int DT, int D>
__global__ __launch_bounds__(256) void lin_step_kernel(LinArgs a) {
    constexpr int QUADS = D / 4, ROWS = 256 / QUADS, N = D / ROWS;
    __shared__ float sum[ROWS][D];
    const int head = blockIdx.x % a.heads, b = blockIdx.x / a.heads, kvh = head / a.group;
    const int c = threadIdx.x % QUADS * 4, r0 = threadIdx.x / QUADS;
    const int64_t at = ((int64_t)b * a.heads + head) * D * D;
    const unsigned short* q = (const unsigned short*)a.Q.p + b * a.Q.ld + head * a.Q.hs;
    const unsigned short* k = (const unsigned short*)a.K.p + b * a.K.ld + kvh * a.K.hs;
    const u2_t vw = *(const u2_t*)((const unsigned short*)a.V.p + b * a.V.ld + kvh * a.V.hs + c);
    f4_t S[N];
#pragma unroll
    for (int i = 0; i < N; ++i) S[i] = *(const f4_t*)(a.s0 + at + (r0 + ROWS * i) * D + c);
    const float lam = __builtin_amdgcn_exp2f(a.log_decay[head] * kLog2e);
    const float v[4] = {attn_unpack<DT>(vw[0], 0), attn_unpack<DT>(vw[0], 1), attn_unpack<DT>(vw[1], 0),
                        attn_unpack<DT>(vw[1], 1)};
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float kk = attn_unpack<DT>(k[r0 + ROWS * i], 0), qq = attn_unpack<DT>(q[r0 + ROWS * i], 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            S[i][e] = __builtin_fmaf(S[i][e], lam, kk * v[e]);
            o[e] = __builtin_fmaf(qq, S[i][e], o[e]);
        }
        *(f4_t*)(a.s1 + at + (r0 + ROWS * i) * D + c) = S[i];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[r0][c + e] = o[e];
    __syncthreads();
    if (threadIdx.x < D / 2) {
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            x += sum[r][2 * threadIdx.x];
            y += sum[r][2 * threadIdx.x + 1];
        }
        *(unsigned*)((char*)a.O + (b * a.ldo + head * a.hso + 2 * threadIdx.x) * 2) = Ty<DT>::pack(x * a.scale, y * a.scale);
    }
}

}  // namespace b2bk
