// Linear attention with a decay for each head: no softmax, and a state
// instead of a cache,
//     S_t = lambda S_{t-1} + k_t v_t^T        (S: D x D, float32)
//     o_t = scale q_t^T S_t.
//
// Prompts go 64 tokens at a time.  With S the state before a chunk and i, j
// its tokens (0 ..),
//     o_i = scale ( lambda^(i+1) q_i^T S + sum_{j<=i} lambda^(i-j) (q_i.k_j) v_j )
//     S'  = lambda^n S + sum_j lambda^(n-1-j) k_j v_j^T
// -- three cascades whose intermediates stay in registers (the relabelled K
// order of the attention kernels):
//   * scores are computed transposed, S^T = K.Q^T, so decayed and rounded
//     they are the operand of V^T.P^T as they lie;
//   * the state's accumulators (lane: value column, registers: key columns,
//     their order set by the order in which the keys' columns are read) are,
//     rounded, the operand of S^T.Q^T as they lie, so the state never leaves
//     its wave's registers;
//   * both end in O^T with one query row a lane, so the factor
//     scale lambda^(i+1) is one multiplication a register.
// Every wave owns 32 value columns: its part of the state (D x 32 floats, 64
// registers at D = 128) and of the output.  Scores are recomputed by each
// wave (24 of its ~90 matrix instructions a chunk) rather than exchanged.
//
// The state is float32 and so are its terms: lambda^(n-1-j) v_j is split into
// parts of the 16-bit type that together hold its 24 bits (bf16: three; fp16:
// two, the second scaled by 2^11), each a pass of matrix instructions with the
// exact k_j.  Only the operands that end in the 16-bit output are rounded to
// its type: the scores and, as q's partner, a copy of the state.
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
    int32_t seg;                // tokens of a segment
    float scale;
};

// lambda^d, d >= 0, from its log2 (exact for d = 0 whatever lambda is)
__device__ __forceinline__ float lin_pow(float g2, int d) {
    return d <= 0 ? 1.f : __builtin_amdgcn_exp2f((float)d * g2);
}

// STATE: only the segments' own states (from zero), for the pass before the
// outputs of sequences that are split.
// LDS: two slots of keys, then values (STATE: two slots), then queries, then
// decays: of the chunk's tokens up to its end, and of the scores.
template <int DT_, int D_, bool STATE_>
struct LinCfg {
    static constexpr int DT = DT_, D = D_, DB = D / 32, WAVES = DB, THREADS = 64 * WAVES, C = 64;
    static constexpr bool STATE = STATE_;
    static constexpr int KS = 2 * DB, TILE = C * DB * 64, FALL = 4 * TILE, DECAYS = FALL + 256;
    static constexpr int LDS_BYTES = DECAYS + (STATE ? 0 : 8192);
    static constexpr int PARTS = DT == DT_BF16 ? 3 : 2;
};

// A transposed fragment of the swizzled key tile: 32 columns of block t,
// K-step ks of its rows; tb[e]: the lane's bases.  Of each 16 columns the
// second and third four trade places: the product's result then has, in lane
// half h and register r, column 16*(r/8) + 8h + r%8 of the block (lin_column),
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
__device__ __forceinline__ int lin_column(int r, int h) { return 16 * (r >> 3) + 8 * h + (r & 7); }
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

template <int DT>
__device__ __forceinline__ float lin_unpack(unsigned w, int hi) {
    if constexpr (DT == DT_BF16) {
        const unsigned x = hi ? (w & 0xFFFF0000u) : (w << 16);
        return __builtin_bit_cast(float, x);
    } else {
        const h2_t v = __builtin_bit_cast(h2_t, w);
        return hi ? (float)v[1] : (float)v[0];
    }
}

// Two values as PARTS 16-bit parts each, packed: their sum holds 24 bits
// (fp16: the second part is scaled by 2^11).
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
            x -= lin_unpack<DT>(out[p], 0);
            y -= lin_unpack<DT>(out[p], 1);
            if constexpr (DT == DT_F16) {
                x *= 2048.f;
                y *= 2048.f;
            }
        }
    }
}

// The exponent e for which the state's largest magnitude times 2^-e is about
// 2^13: fp16 copies of larger or much smaller states would leave its range.
// Uniform over the wave; 0 for states that are in range as they are.
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
    if (!(m > 0.f) || m > 3e38f) return 0;
    return __builtin_amdgcn_readfirstlane(__builtin_amdgcn_frexp_expf(m) - 13);
}

template <class C>
__device__ __forceinline__ void lin_body(const LinArgs& a) {
    __shared__ __attribute__((aligned(1024))) unsigned char lds[C::LDS_BYTES];
    using M = Ty32<C::DT>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int h = lane >> 5, m = lane & 31;
    const int head = blockIdx.x % a.heads, tile = blockIdx.x / a.heads, kvh = head / a.group;
    SeqTile w;
    // (a sequence without tokens counts as one empty segment: its state still passes through)
    if (!find_tile(a.cu, nullptr, a.seqs, (int)a.rows, 0, 1, a.seg, 1, tile, &w)) return;
    const bool last = w.local + 1 == w.tiles;
    if (C::STATE && last) return;       // nobody reads what follows the last segment
    const int64_t row0 = w.q0 + (int64_t)w.local * a.seg;
    const int n = last ? w.nq - w.local * a.seg : a.seg;
    const float g2 = a.log_decay[head] * kLog2e;

    // this wave's columns of the state
    f16x_t S[C::DB];
    const int col = 32 * wave + m;
    auto state_at = [&](float* base, int64_t slot) { return base + ((slot * a.heads + head) * C::D) * C::D + col; };
    const float* from = nullptr;
    if constexpr (!C::STATE) {
        if (w.tiles > 1) from = state_at(a.part, tile);
        else if (a.s0) from = state_at(const_cast<float*>(a.s0), w.seq);
    }
#pragma unroll
    for (int t = 0; t < C::DB; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) S[t][r] = from ? from[(32 * t + lin_column(r, h)) * C::D] : 0.f;

    const int chunks = (n + C::C - 1) / C::C;
    const int64_t qat = (int64_t)head * a.Q.hs, kat = (int64_t)kvh * a.K.hs, vat = (int64_t)kvh * a.V.hs;
    auto copy = [&](const AttnRows& x, int64_t at, int c, int slot, auto SWZ) __attribute__((always_inline)) {
        const auto rs = attn_rsrc(x.p, row0 + (int64_t)c * C::C, x.ld, at, n - c * C::C < C::C ? n - c * C::C : C::C, C::D);
#pragma unroll
        for (int rg = wave; rg < 4; rg += C::WAVES)
            attn_copy<C::DB, C::C, SWZ.value>(lds + slot * C::TILE, rs, (int)x.ld * 2, C::D, rg, lane);
    };
    auto copy_k = [&](int c) { copy(a.K, kat, c, c & 1, std::true_type{}); };
    auto copy_v = [&](int c) { copy(a.V, vat, c, C::STATE ? 2 + (c & 1) : 2, std::false_type{}); };
    auto copy_q = [&](int c) { copy(a.Q, qat, c, 3, std::true_type{}); };
    const int kb[2] = {attn_kbase(lane, 0), attn_kbase(lane, 1)};
    int tb[2];
    lin_tbase(lane, tb);
    auto rows32 = [&](int off, int s) __attribute__((always_inline)) {     // a fragment of 32 rows, K-step s
        return *(const u4_t*)(lds + off + kb[s & 1] + (s >> 1) * C::C * 64);
    };
    const int vb = attn_vbase(lane);
    // decays of the scores: of a pair of tokens in the same half of the chunk
    // (0 where the key comes later) and of a query in the second half with a
    // key in the first
    // -- in LDS, 16 of each a lane: in registers they would cost two waves a SIMD
    float into[2];
    if constexpr (!C::STATE) {
        for (int g = wave; g < 8; g += C::WAVES) {
            f4_t d;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = 8 * (g & 3) + 4 * h + r;
                d[r] = g >= 4 ? a.scale * lin_pow(g2, 32 + m - j) : (j > m ? 0.f : a.scale * lin_pow(g2, m - j));
            }
            *(f4_t*)(lds + C::DECAYS + g * 1024 + lane * 16) = d;
        }
        into[0] = a.scale * lin_pow(g2, m + 1);
        into[1] = a.scale * lin_pow(g2, m + 33);
    }
    float* fall = (float*)(lds + C::FALL);       // lambda^(n-1-j) of token j of the chunk
    if (wave == 0) fall[lane] = lin_pow(g2, 63 - lane);

    if (chunks > 0) {
        copy_k(0);
        copy_v(0);
        if constexpr (!C::STATE) copy_q(0);
    }
    for (int c = 0; c < chunks; ++c) {
        barrier_vm<0>();       // chunk c is in LDS, and everyone is done with chunk c - 1
        if (c + 1 < chunks) copy_k(c + 1);
        const unsigned char* kt = lds + (c & 1) * C::TILE;
        const int left = n - c * C::C < C::C ? n - c * C::C : C::C;
        u4_t v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = attn_vfrag<C::C>(lds + (C::STATE ? 2 + (c & 1) : 2) * C::TILE, vb, wave, k);
        if constexpr (C::STATE) {
            if (c + 1 < chunks) copy_v(c + 1);
        } else {
            // the state as an operand
            u4_t sp[C::KS];
            int e = 0;
            if constexpr (C::DT == DT_F16) e = lin_exponent(S);
            if (e != 0) {
                const float down = __builtin_ldexpf(1.f, -e);
#pragma unroll
                for (int s = 0; s < C::KS; ++s) {
                    f16x_t x = S[s >> 1];
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[r] *= down;
                    sp[s] = attn_pack<C::DT>(x, s & 1);
                }
            } else {
#pragma unroll
                for (int s = 0; s < C::KS; ++s) sp[s] = attn_pack<C::DT>(S[s >> 1], s & 1);
            }
            const float up = __builtin_ldexpf(1.f, e);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                u4_t q[C::KS];
#pragma unroll
                for (int s = 0; s < C::KS; ++s) q[s] = rows32(3 * C::TILE + i * 2048, s);
                if (i == 1) {
                    // the last chunk's tokens count up to its own end
                    if (left < C::C && wave == 0) fall[lane] = lin_pow(g2, left - 1 - lane);
                    barrier_lds();       // everyone has read this chunk's values and queries
                    if (c + 1 < chunks) {
                        copy_v(c + 1);
                        copy_q(c + 1);
                    }
                }
                // from the state
                f16x_t o = f16x_t{};
#pragma unroll
                for (int s = 0; s < C::KS; ++s) o = M::mma(sp[s], q[s], o);
                const float f = into[i] * up;
#pragma unroll
                for (int r = 0; r < 16; ++r) o[r] *= f;
                // from the chunk's own tokens
#pragma unroll
                for (int k = 0; k <= i; ++k) {
                    f16x_t p = f16x_t{};
#pragma unroll
                    for (int s = 0; s < C::KS; ++s) p = M::mma(rows32((c & 1) * C::TILE + k * 2048, s), q[s], p);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const f4_t d = *(const f4_t*)(lds + C::DECAYS + ((i == k ? 0 : 4) + g) * 1024 + lane * 16);
#pragma unroll
                        for (int r = 0; r < 4; ++r) p[4 * g + r] *= d[r];
                    }
#pragma unroll
                    for (int s = 0; s < 2; ++s) o = M::mma(v[2 * k + s], attn_pack<C::DT>(p, s), o);
                }
                const int row = 32 * i + m;
                char* op = (char*)a.O + ((row0 + (int64_t)c * C::C + row) * a.ldo + (int64_t)head * a.hso + 32 * wave) * 2;
#pragma unroll
                for (int q4 = 0; q4 < 4; q4 += 2) {
                    unsigned x0 = Ty<C::DT>::pack(o[4 * q4], o[4 * q4 + 1]);
                    unsigned x1 = Ty<C::DT>::pack(o[4 * q4 + 2], o[4 * q4 + 3]);
                    unsigned y0 = Ty<C::DT>::pack(o[4 * q4 + 4], o[4 * q4 + 5]);
                    unsigned y1 = Ty<C::DT>::pack(o[4 * q4 + 6], o[4 * q4 + 7]);
                    swap32(x0, y0);
                    swap32(x1, y1);
                    if (row < left) *(u4_t*)(op + 16 * (q4 + h)) = u4_t{x0, x1, y0, y1};
                }
                __builtin_amdgcn_sched_barrier(0);   // the two halves' registers in turn
            }
        }
        // the state after the chunk
        u4_t vp[C::PARTS][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const f4_t w = *(const f4_t*)(fall + 16 * k + 8 * x + 4 * h);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const unsigned two = v[k][2 * x + y];
                    unsigned out[C::PARTS];
                    lin_split<C::DT>(lin_unpack<C::DT>(two, 0) * w[2 * y], lin_unpack<C::DT>(two, 1) * w[2 * y + 1], out);
#pragma unroll
                    for (int p = 0; p < C::PARTS; ++p) vp[p][k][2 * x + y] = out[p];
                }
            }
        const float keep = lin_pow(g2, left);
#pragma unroll
        for (int t = 0; t < C::DB; ++t) {
            u4_t f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = lin_tfrag<C::C>(kt, tb, t, k);
            if constexpr (C::DT == DT_F16) {
                f16x_t low = f16x_t{};
#pragma unroll
                for (int k = 0; k < 4; ++k) low = M::mma(f[k], vp[1][k], low);
#pragma unroll
                for (int r = 0; r < 16; ++r) S[t][r] = __builtin_fmaf(low[r], 1.f / 2048, S[t][r] * keep);
#pragma unroll
                for (int k = 0; k < 4; ++k) S[t] = M::mma(f[k], vp[0][k], S[t]);
            } else {
#pragma unroll
                for (int r = 0; r < 16; ++r) S[t][r] *= keep;
#pragma unroll
                for (int p = C::PARTS - 1; p >= 0; --p)
#pragma unroll
                    for (int k = 0; k < 4; ++k) S[t] = M::mma(f[k], vp[p][k], S[t]);
            }
        }
    }
    float* to = nullptr;
    if constexpr (C::STATE) to = state_at(a.part, tile);
    else if (last && a.s1) to = state_at(a.s1, w.seq);
    if (to)
#pragma unroll
        for (int t = 0; t < C::DB; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) to[(32 * t + lin_column(r, h)) * C::D] = S[t][r];
}

template <class C>
__global__ __launch_bounds__(C::THREADS, 2) void lin_kernel(LinArgs a) {
    lin_body<C>(a);
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
    const float v[4] = {lin_unpack<DT>(vw[0], 0), lin_unpack<DT>(vw[0], 1), lin_unpack<DT>(vw[1], 0),
                        lin_unpack<DT>(vw[1], 1)};
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float kk = lin_unpack<DT>(k[r0 + ROWS * i], 0), qq = lin_unpack<DT>(q[r0 + ROWS * i], 0);
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
