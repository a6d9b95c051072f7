// Causal attention whose keys lie in the pages of a cache, and attention under
// a window with the first keys still visible.
//
// The products, the softmax and their layouts are attn.hpp's: scores transposed
// on v_mfma_f32_32x32x16, a query row a lane, the rounded probabilities the
// second product's operand as they lie.  What differs is which keys a row meets
// and where they are:
//
//   Pages.  Key j of sequence s is row j % size of page table[s][j / size].  Loads
//   write LDS directly, 16 rows of 64 bytes each.  Pages of a multiple of 16 keys:
//   the 16 rows lie in one page, whose address is one scalar calculation and a
//   buffer resource that ends at the sequence's last key (many rows, whose time is
//   instructions: 2048 rows behind 16384 keys 404 us -> 362; the few rows' kernel
//   waits for memory and was faster without the scalar chain, 215 us against 223
//   when its 64 requests took that, 201 now).
//   Else, as pages of other sizes may end anywhere, every lane works out the address
//   (64 bits) of the 16 bytes that it moves, and those behind the last key come from
//   a block of zeros.  Either way what a page holds behind a sequence's keys may be
//   anything, NaN too.  The table's entries for a tile are asked for a tile ahead.
//
//   Window.  The row in place p sees keys p - window + 1 .. p and the first
//   `sinks`: 128 rows' tiles are those of the sinks and those from the first
//   row's window on, one range with a gap.  Only tiles at the range's borders
//   are masked.
//
// Work is cut on the device, where the lengths are.  A (sequence, tile of 128
// rows, key head) of T key tiles is cut into ceil(T / L) parts, with L the larger
// of `least` and the whole call's key tiles over the workgroups that it should
// have: no chain of tiles is longer than that, whatever the lengths, and a
// captured graph replays with new ones.  Sequences of up to 32 rows, whose partial
// results are small and whose time is the bytes of their keys, are cut finer, into
// parts of max(L / 4, min(4 L, 32), 8), of this L without `least`: four times as fine
// where there is much work, 32 tiles from L = 8 on, less where there is little.
// Since sum ceil(T / L) <= items + sum T / L, four times the sum for few rows, the
// host knows the grid's size, and since a cut item has at most twice its T / L
// parts, the partial results' as well: 32 rows a granule, one of a part of few
// rows, four of a tile's.
#pragma once
#include "attn.hpp"

namespace b2bk {

struct Pages {
    const void* p;
    int64_t ps, ld, hs;     // from page to page, row to row, head to head
};

struct KeyArgs : AttnArgs {
    Pages pk, pv;
    const int32_t* table;   // [seqs, width], rows table_ld apart
    int64_t table_ld;
    FastDiv page;           // keys a page
    int32_t pages, window, sinks;
    int32_t split, least;   // whether items may be cut: those of more than `least` key tiles
    float per;              // key heads over the workgroups that a call should have
    int32_t granules;       // of partial results, a key head
    int32_t subs;           // granules of a tile that the join looks for (1: no sequence has more than 32 rows)
    int32_t spread;         // whether a key head's workgroups go over all XCDs
};

constexpr int kKeyRows = 128;     // rows of a tile

// 16 bytes a lane from an address of its own to LDS (lane i -> dst + 16 i),
// issued and waited for as lds_dma16's.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_dma16_from(const unsigned char* dst, const char* p) {
    const unsigned a = (unsigned)(uintptr_t)(lds_ptr_t)dst;
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(a), "v"(p) : "memory", "m0");
}
// The same of 4 bytes a lane.
__device__ __forceinline__ void lds_dma4_from(const unsigned char* dst, const void* p) {
    const unsigned a = (unsigned)(uintptr_t)(lds_ptr_t)dst;
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, off" : : "s"(a), "v"(p) : "memory", "m0");
}
#pragma clang diagnostic pop

// what places behind a sequence's last key and columns past the head's read
__device__ __attribute__((aligned(256))) const unsigned char kZeros[256] = {};

// ---------------------------------------------------------------------------
// Where a workgroup works
// ---------------------------------------------------------------------------
struct KeyItem {
    int seq, tile, part, parts;
    int granule, per_part;              // the tile's first, and those of a part
    int q0, nq, k0, nk;
    int tiles;
};

__device__ __forceinline__ float lanes_total(float x) {
    auto up = [&](int y) { x += __builtin_bit_cast(float, y); };
    auto me = [&] { return __builtin_bit_cast(int, x); };
    up(__builtin_amdgcn_update_dpp(0, me(), 0x111, 0xf, 0xf, false));
    up(__builtin_amdgcn_update_dpp(0, me(), 0x112, 0xf, 0xf, false));
    up(__builtin_amdgcn_update_dpp(0, me(), 0x114, 0xf, 0xf, false));
    up(__builtin_amdgcn_update_dpp(0, me(), 0x118, 0xf, 0xf, false));
    up(__builtin_amdgcn_update_dpp(0, me(), 0x142, 0xa, 0xf, false));
    up(__builtin_amdgcn_update_dpp(0, me(), 0x143, 0xc, 0xf, false));
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(me(), 63));
}

// The item (JOIN: the tile, whatever its parts) number u, sequences 64 at a time.
template <bool PAGED, bool WIN, bool JOIN>
__device__ __forceinline__ bool find_item(const KeyArgs& a, int u, KeyItem* out) {
    const int lane = threadIdx.x & 63, group = a.group.d;
    int q0, n, k0, nk, tiles, span;
    auto load = [&](int s0) __attribute__((always_inline)) {
        const int s = s0 + lane;
        q0 = n = k0 = nk = 0;
        if (s < a.seqs) {
            if (a.cu_q) seq_range(a.cu_q, s, (int)a.rows, &q0, &n);
            else q0 = s, n = 1;
            if constexpr (PAGED) {
                nk = a.lens[s];
                nk = nk < 0 ? 0 : (nk > (int)a.keys ? (int)a.keys : nk);
            } else {
                seq_range(a.cu_k, s, (int)a.keys, &k0, &nk);
            }
        }
        tiles = (int)(((unsigned)n * (unsigned)group + kKeyRows - 1) / kKeyRows);
        span = (nk + 31) >> 5;              // key tiles of the tile that has the most, or a few more
        if constexpr (WIN) {
            const int tokens = a.group(kKeyRows + group - 2) + 1;
            const int w = ((a.window + (n < tokens ? n : tokens)) >> 5) + ((a.sinks + 31) >> 5) + 2;
            span = span < w ? span : w;
        }
    };
    load(0);
    int most = 1 << 30, fine = 1 << 30;      // key tiles of a part; of sequences of few rows
    if (a.split) {
        double work = (double)tiles * span;
        for (int s0 = 64; s0 < a.seqs; s0 += 64) {
            load(s0);
            work += (double)tiles * span;
        }
        if (a.seqs > 64) load(0);
        // (a thousandth more than the sum, so that its rounding makes no part too many)
        const float l = ceilf(lanes_total((float)work) * 1.001f * a.per);
        most = l > (float)(1 << 30) ? 1 << 30 : (int)l;
        // Of few rows: the less work there is, the finer, for a wave's chain of tiles is
        // then all the time (one request of 2048 keys, 8 key heads: 19.5 us in parts of 32
        // tiles, 15.1 of 16, 12.9 of 8; 16 requests: 35.5, 37.2, 40.0).
        const int some = most < 8 ? 4 * most : 32;
        fine = (most + 3) >> 2;
        fine = fine < some ? some : fine;
        fine = fine < 8 ? 8 : fine;
        most = most < a.least ? a.least : most;
    }
    int before = 0, used = 0;
    for (int s0 = 0;;) {
        const bool few = (unsigned)n * (unsigned)group <= 32;
        const int l = few ? fine : most;
        const int parts = a.split && span > a.least && span > l ? (int)(((unsigned)span + (unsigned)l - 1) / (unsigned)l) : 1;
        const int per_part = few ? 1 : kKeyRows / 32;
        const int mine = JOIN ? tiles : tiles * parts, cut = parts > 1 ? tiles * parts * per_part : 0;
        const int sum = lanes_sum(mine), cuts = lanes_sum(cut);
        const unsigned long long hit = __ballot(before + sum > u);
        if (hit) {
            const int at = __ffsll(hit) - 1;
            const int local = u - before - (__builtin_amdgcn_readlane(sum, at) - __builtin_amdgcn_readlane(mine, at));
            // (starts out of order may name more tiles than there can be rows: what the grid
            // and the workspace were not made for is left out)
            if ((unsigned)local >= (unsigned)__builtin_amdgcn_readlane(mine, at)) return false;
            out->seq = s0 + at;
            out->parts = __builtin_amdgcn_readlane(parts, at);
            out->per_part = __builtin_amdgcn_readlane(per_part, at);
            out->tiles = __builtin_amdgcn_readlane(tiles, at);
            out->tile = JOIN || out->parts == 1 ? local : (int)((unsigned)local / (unsigned)out->parts);
            out->part = JOIN ? 0 : local - out->tile * out->parts;
            out->granule = used + __builtin_amdgcn_readlane(cuts, at) - __builtin_amdgcn_readlane(cut, at) +
                           out->tile * out->parts * out->per_part;
            out->q0 = __builtin_amdgcn_readlane(q0, at);
            out->nq = __builtin_amdgcn_readlane(n, at);
            out->k0 = __builtin_amdgcn_readlane(k0, at);
            out->nk = __builtin_amdgcn_readlane(nk, at);
            return out->parts == 1 || out->granule + out->parts * out->per_part <= a.granules;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
        used += __builtin_amdgcn_readlane(cuts, 63);
        s0 += 64;
        if (s0 >= a.seqs) return false;
        load(s0);
    }
}

// ---------------------------------------------------------------------------
// One item's geometry
// ---------------------------------------------------------------------------
// Where keys lie: side by side, in pages of a multiple of 16 keys, in pages of any size.
enum { KEYS_PACKED, KEYS_PAGES16, KEYS_PAGES };

// FEW: for calls whose sequences have few rows, with LDS for twice the keys in flight.
template <int DT_, int DB_, int WHERE_, bool WIN_, bool FEW_ = false>
struct KeyCfg {
    static constexpr int DT = DT_, DB = DB_, WAVES = 4, THREADS = 64 * WAVES, BM = kKeyRows, BN = 32, WHERE = WHERE_;
    static constexpr bool PAGED = WHERE != KEYS_PACKED, WIN = WIN_, FEW = FEW_;
    static constexpr int KS = 2 * DB;                   // K-steps of the first product
    static constexpr int TILE = BN * DB * 64;           // a tile of keys (or values) in LDS
    static constexpr int MINE = FEW ? 2 * TILE + 256 : TILE;     // a wave's LDS where waves take different keys
    static constexpr int JOIN = WAVES * MINE;           // behind it: the waves' maxima and sums
    static constexpr int QUERIES = 2 * TILE;            // the waves' queries on their way: the second slot of keys and behind it
    static constexpr int LDS_BYTES = QUERIES + WAVES * TILE > JOIN + 2 * WAVES * 32 * 4 ? QUERIES + WAVES * TILE
                                                                                        : JOIN + 2 * WAVES * 32 * 4;
    // Workgroups a compute unit, by registers: 110 to 164 of them.  (Heads of 65 to 96 held to the 128 of four spill 3
    // to 21 but for pages of whole groups under a window, which gain nothing by it: 24 heads of 96 on 4, 1464 rows in
    // 4 chunks and 36 single tokens 66.5 us with either bound, 2048 rows behind 30000 keys 65.1; heads of up to 64 take 114.)
    static constexpr int PER_CU = FEW ? 2 : 3;
    static_assert(BM == 32 * WAVES, "many rows: 32 a wave");
    static_assert(!FEW || PAGED, "few rows: pages");
};

// Which key tiles the rows of a tile meet: number i of [i0, i1) is tile
// i < sink_tiles ? i : i + gap.
template <class C>
struct KeyTile {
    const KeyArgs& a;
    const KeyItem& w;
    int kvh, row0, rows, shift;      // rows: the sequence's; row r is token r / group, in place r / group + shift
    int i0, i1, sink_tiles, gap;

    __device__ __forceinline__ KeyTile(const KeyArgs& args, const KeyItem& item, int head) : a(args), w(item), kvh(head) {
        row0 = (w.tiles - 1 - w.tile) * C::BM;      // the last rows see the most keys: they start first
        rows = w.nq * a.group.d;
        shift = w.nk - w.nq;
        const int last = (row0 + C::BM < rows ? row0 + C::BM : rows) - 1;
        const int end = (sees(last) + C::BN - 1) / C::BN;
        int n = end;
        sink_tiles = end;
        gap = 0;
        if constexpr (C::WIN) {
            const int lo = from(row0), first = lo > 0 ? lo / C::BN : 0, s = (a.sinks + C::BN - 1) / C::BN;
            if (first > s && end > first) {
                sink_tiles = s;
                gap = first - s;
                n = end - gap;
            }
        }
        i0 = 0;
        i1 = n;
        if (w.parts > 1) {
            const int whole = (int)((unsigned)n / (unsigned)w.parts), rest = n - whole * w.parts;
            i0 = whole * w.part + (int)((unsigned)(rest * w.part) / (unsigned)w.parts);
            i1 = whole * (w.part + 1) + (int)((unsigned)(rest * (w.part + 1)) / (unsigned)w.parts);
        }
    }
    __device__ __forceinline__ int tile(int i) const { return C::WIN && i >= sink_tiles ? i + gap : i; }
    // keys that row r sees end here (places 0 .. sees - 1) ...
    __device__ __forceinline__ int sees(int r) const {
        if (r >= rows) return 0;
        const int n = a.group(r) + 1 + shift;
        return n < 0 ? 0 : n;
    }
    // ... and begin here, the sinks apart
    __device__ __forceinline__ int from(int r) const {
        // (a window is 2^30 at most)
        return a.group(r) + 1 + shift - a.window;
    }
    __device__ __forceinline__ int entry(int key) const {
        key = key < w.nk ? key : w.nk - 1;
        return a.table[w.seq * a.table_ld + a.page(key)];
    }
    // 16-byte piece `chunk` of key `key`'s row, whose page the table's entry names
    __device__ __forceinline__ const char* row_at(const Pages& x, int key, int entry, int chunk) const {
        const int in = key - a.page(key) * a.page.d;
        const int pg = entry < 0 ? 0 : (entry < a.pages ? entry : a.pages - 1);
        return (const char*)x.p + (pg * x.ps + in * x.ld + kvh * x.hs + 8 * chunk) * 2;
    }
    // one key's row, wherever it lies
    __device__ __forceinline__ const char* key_row(bool values, int key) const {
        if constexpr (C::PAGED) return row_at(values ? a.pv : a.pk, key, entry(key), 0);
        const AttnRows& x = values ? a.V : a.K;
        return (const char*)x.p + (((int64_t)w.k0 + key) * x.ld + kvh * x.hs) * 2;
    }
    // Copies row group rg (16 rows) of a tile of a cache, keys with their chunks
    // swizzled as attn_copy's, every lane from an address of its own; e: the
    // lane's table entry.
    template <bool VALUES>
    __device__ __forceinline__ void copy_lanes(const unsigned char* dst, int t, int rg, int e, int lane) const {
        const int row = 16 * rg + (lane >> 2), key = t * C::BN + row;
        const int chunk = VALUES ? (lane & 3) : ((lane & 3) ^ ((row >> 2) & 3));
        const bool in = key < w.nk;
        const char* p = row_at(VALUES ? a.pv : a.pk, key, e, chunk);
#pragma unroll
        for (int b = 0; b < C::DB; ++b)
            lds_dma16_from(dst + b * C::BN * 64 + rg * 1024, in && 32 * b + 8 * chunk < a.dim ? p + 64 * b : (const char*)kZeros);
    }
    // The same of keys side by side.
    template <bool VALUES>
    __device__ __forceinline__ void copy_packed(const unsigned char* dst, int t, int rg, int lane) const {
        const AttnRows& x = VALUES ? a.V : a.K;
        const int n = w.nk - t * C::BN < C::BN ? w.nk - t * C::BN : C::BN;
        const auto rs = attn_rsrc(x.p, (int64_t)w.k0 + (int64_t)t * C::BN, x.ld, (int64_t)kvh * x.hs, n, a.dim);
        attn_copy<C::DB, C::BN, !VALUES>(dst, rs, (int)x.ld * 2, a.dim, rg, lane);
    }
    // Copies a lane's 16-byte pieces of query row rr, one of group rg (16 rows) of a
    // wave's, laid out as keys.
    __device__ __forceinline__ void copy_queries(const unsigned char* dst, int rr, int rg, int lane) const {
        const int chunk = (lane & 3) ^ ((lane >> 4) & 3), pos = a.group(rr), head = kvh * a.group.d + (rr - pos * a.group.d);
        const char* p = (const char*)a.Q.p + ((w.q0 + pos) * a.Q.ld + head * a.Q.hs + 8 * chunk) * 2;
#pragma unroll
        for (int b = 0; b < C::DB; ++b)
            lds_dma16_from(dst + b * C::BN * 64 + rg * 1024, rr < rows && 32 * b + 8 * chunk < a.dim ? p + 64 * b : (const char*)kZeros);
    }
    // lane's table entry for row group rg of tile t
    __device__ __forceinline__ int entry_of(int t, int rg, int lane) const {
        if constexpr (C::PAGED) return entry(t * C::BN + 16 * rg + (lane >> 2));
        return 0;
    }
    __device__ __forceinline__ int64_t part_row(int rr) const {
        const int r = rr - row0;
        return ((int64_t)(w.granule + w.part * w.per_part + (r >> 5)) * a.kv_heads.d + kvh) * 32 + (r & 31);
    }
};

// Whether a lane's row sees key c + 4 (lane / 32) of a tile; lim, lo and sinks
// are counted from the tile's first key, less 4 for the upper half of the lanes.
template <bool WIN>
__device__ __forceinline__ bool key_seen(int c, int lim, int lo, int sinks) {
    return c < lim && (!WIN || c >= lo || c < sinks);
}

template <bool WIN>
__device__ __forceinline__ void key_mask(f16x_t& s, int lim, int lo, int sinks) {
#pragma unroll
    for (int r = 0; r < 16; ++r)
        if (!key_seen<WIN>(8 * (r >> 2) + (r & 3), lim, lo, sinks)) s[r] = -__builtin_inff();
}

// The lane's number, from which nothing that was worked out before is kept: behind a
// loop it costs instructions, not registers inside it.
__device__ __forceinline__ int lane_again() {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    return lane;
}

// attn_move_max, the two halves' maxima joined by a swap alone.
template <int NO>
__device__ __forceinline__ void key_move_max(float mx, RowState& st, f16x_t (&o)[NO], float sc) {
    unsigned x = __builtin_bit_cast(unsigned, mx), y = x;
    swap32(x, y);       // x: the low half's in all lanes, y: the high half's
    mx = __builtin_fmaxf(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y)) * sc;
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

// Infinities and NaN among the values (see attn_finite): the wave's rows again,
// straight from memory, tiles i0, i0 + step, ... below i1, values that are not
// finite left out.  Then the rows that see such a value get it: a product of
// ones (where a key is seen) with ones (where its value is +inf or NaN, then
// -inf or NaN) counts them for every row and column, whatever the rows see.
// Few registers before speed.
template <class C>
__device__ __forceinline__ void key_again(const KeyTile<C>& k, f16x_t (&o)[C::DB], const RowState& st, int rr, int i0, int step,
                                          int lane) {
    using M = Ty32<C::DT>;
    constexpr unsigned kExp = C::DT == DT_BF16 ? 0x7F80 : 0x7C00, kOne = C::DT == DT_BF16 ? 0x3F80 : 0x3C00;
    const KeyArgs& a = k.a;
    const int m = lane & 31, h = lane >> 5, nk = k.w.nk;
    const int pos = a.group(rr), head = k.kvh * a.group.d + (rr - pos * a.group.d);
    const int lim = k.sees(rr) - 4 * h, lo = C::WIN ? k.from(rr) - 4 * h : 0;
    // column 32b + m of 8 keys' values; kind 0: the finite ones, 1, 2: ones in place of the others
    auto values = [&](int t, int ks, int b, int kind) __attribute__((always_inline)) {
        u4_t x = {0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int at = t * C::BN + 16 * ks + 8 * (u >> 2) + 4 * h + (u & 3), c = 32 * b + m;
            unsigned v = 0;
            if (at < nk && c < a.dim) v = *(const unsigned short*)(k.key_row(true, at) + 2 * c);
            const bool odd = (v & kExp) == kExp, nan = odd && (v & 0x7FFF & ~kExp);
            if (kind == 0) v = odd ? 0 : v;
            else v = nan || (odd && (int)(v >> 15) == kind - 1) ? kOne : 0;
            x[u >> 1] |= v << (16 * (u & 1));
        }
        return x;
    };
#pragma unroll
    for (int b = 0; b < C::DB; ++b) o[b] = f16x_t{};
    for (int i = i0; i < k.i1; i += step) {
        const int t = k.tile(i), key = t * C::BN + m;
        const char* kp = key < nk ? k.key_row(false, key) : (const char*)kZeros;
        f16x_t s = f16x_t{};
#pragma unroll 1
        for (int j = 0; j < C::KS; ++j) {
            const bool in = 16 * j + 8 * h < a.dim;
            u4_t x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
            if (in && key < nk) x = *(const u4_t*)(kp + 32 * j + 16 * h);
            if (in && rr < k.rows)
                y = *(const u4_t*)((const char*)a.Q.p + ((k.w.q0 + pos) * a.Q.ld + (int64_t)head * a.Q.hs + 16 * j + 8 * h) * 2);
            s = M::mma(x, y, s);
        }
        key_mask<C::WIN>(s, lim - t * C::BN, lo - t * C::BN, a.sinks - 4 * h - t * C::BN);
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], a.sc, -st.m));
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const u4_t p = attn_pack<C::DT>(s, ks);
#pragma unroll
            for (int b = 0; b < C::DB; ++b) {
                o[b] = M::mma(values(t, ks, b, 0), p, o[b]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
#pragma unroll
    for (int b = 0; b < C::DB; ++b)
#pragma unroll 1
        for (int kind = 1; kind <= 2; ++kind) {
            f16x_t n = f16x_t{};
            for (int i = i0; i < k.i1; i += step) {
                const int t = k.tile(i), x = t * C::BN;
#pragma unroll 1
                for (int ks = 0; ks < 2; ++ks) {
                    u4_t p = {0, 0, 0, 0};
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const int c = 16 * ks + 8 * (u >> 2) + (u & 3);
                        if (key_seen<C::WIN>(c, lim - x, lo - x, a.sinks - 4 * h - x)) p[u >> 1] |= kOne << (16 * (u & 1));
                    }
                    n = M::mma(values(t, ks, b, kind), p, n);
                }
            }
            const float give = kind == 1 ? __builtin_inff() : -__builtin_inff();
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (n[r] != 0.f) o[b][r] += give;
        }
}

// ---------------------------------------------------------------------------
// Many rows: 32 a wave, the key tiles shared (attn_tile_body's scheme)
// ---------------------------------------------------------------------------
// Measured (bf16, 32 heads of 128 on 8 key heads): 32768 tokens under a window of
// 4096 in 1.77 to 1.98 ms by the card, 1040 to 1165 TFLOP/s of the 1230 to 1290 that a
// product of 8192^3 reaches (matrix cores busy 0.74 of the cycles at a clock that power
// holds at 1.5 to 1.6 GHz); 8001 tokens in 17 sequences under a window of 512 in 64 to 68
// us, 59 where the caches hold all of it: of a workgroup's 37 thousand cycles some 4.3
// went to finding its place, 7.2 to its first keys and queries (before these came
// through LDS), 22.6 to 10 tiles and 2.9 to its output; 2048 rows of 4 sequences behind
// up to 16384 keys in pages of 64 in 360 to 380 us and 7 for the join (matrix cores
// busy 0.59).  Tile i's probabilities worked out under tile i + 1's scores, which
// costs no LDS but 16 registers, was slower (1858 us -> 1925 and 380 -> 393): what
// waves do side by side covers that already.
template <class C>
__device__ __forceinline__ void key_tile_body(const KeyTile<C>& k, unsigned char* lds) {
    using M = Ty32<C::DT>;
    const KeyArgs& a = k.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wrow = k.row0 + 32 * wave, rr = wrow + (lane & 31), h = lane >> 5;
    const int lim = k.sees(rr) - 4 * h, lo = C::WIN ? k.from(rr) - 4 * h : 0;
    u4_t q[C::KS];
    f16x_t o[C::DB];
    RowState st;
    st.init();
#pragma unroll
    for (int b = 0; b < C::DB; ++b) o[b] = f16x_t{};
    // tiles below `clear` are full and end where every row of the wave sees (lanes past the
    // last row are not looked at: a wave that masked all its tiles for them took a third
    // longer, and the launch with it); from `done` on none sees any; under a window rows
    // see nothing of tiles that end at `dark` or before, everything from `open` on
    const int clear = wrow < k.rows ? k.sees(wrow) / C::BN : 0;
    const int wlast = (wrow + 32 < k.rows ? wrow + 32 : k.rows) - 1;
    const int done = wrow < k.rows ? (k.sees(wlast) + C::BN - 1) / C::BN : 0;
    const int dark = C::WIN ? k.from(wrow) : 0, open = C::WIN ? k.from(wlast) : 0;
    // Two waves copy the keys, two the values, a group of 16 rows each.  Where a
    // group's rows are evenly spaced (keys side by side, pages of whole groups) its
    // address is scalar, and all but the table's entry is worked out early.
    constexpr bool EVEN = C::WHERE != KEYS_PAGES;
    const bool keys = wave < 2;
    const int rg = wave & 1;
    const Pages src = C::PAGED ? (keys ? a.pk : a.pv)
                               : Pages{keys ? a.K.p : a.V.p, 0, keys ? a.K.ld : a.V.ld, keys ? a.K.hs : a.V.hs};
    const char* src0 = (const char*)src.p + (C::PAGED ? 0 : k.w.k0 * src.ld * 2) + k.kvh * src.hs * 2;
    const uint32_t ld2 = (uint32_t)src.ld * 2, ps2 = (uint32_t)src.ps * 2;     // (pages of whole groups: 4 GB apart at most)
    int off[C::DB];         // a lane's 16 bytes of each block of 32 columns (past the head: past the resource)
    if constexpr (EVEN) {
        const int chunk = keys ? (lane & 3) ^ ((lane >> 4) & 3) : lane & 3;      // swizzled as attn_copy's
#pragma unroll
        for (int b = 0; b < C::DB; ++b) off[b] = 32 * b + 8 * chunk < a.dim ? (lane >> 2) * (int)ld2 + 16 * chunk + 64 * b : -16;
    }
    struct {
        int e;              // the next tile's entry ...
        uint32_t in;        // ... and how far into the page its first row lies
    } next = {0, 0};
    auto look = [&](int i) __attribute__((always_inline)) {
        if constexpr (C::WHERE == KEYS_PAGES16) {
            const int key = k.tile(i) * C::BN + 16 * rg, pg = a.page(key < k.w.nk ? key : k.w.nk - 1);
            next.e = a.table[k.w.seq * a.table_ld + pg];
            next.in = (uint32_t)(key - pg * a.page.d) * ld2;
        } else {
            next.e = k.entry_of(k.tile(i), rg, lane);
        }
    };
    // WHOLE: all of the tile's rows are keys.
    auto copy = [&](int i, int slot, auto WHOLE) __attribute__((always_inline)) {
        const unsigned char* dst = lds + (keys ? 0 : C::TILE) + slot;
        const int t = k.tile(i);
        if constexpr (EVEN) {
            const int key = t * C::BN + 16 * rg, n = WHOLE.value ? 16 : k.w.nk - key;
            const char* p = src0;
            if constexpr (C::PAGED) {
                const int e = __builtin_amdgcn_readfirstlane(next.e), pg = e < 0 ? 0 : (e < a.pages ? e : a.pages - 1);
                p += (uint64_t)(uint32_t)pg * ps2 + next.in;
            } else {
                p += (uint64_t)(uint32_t)key * ld2;
            }
            const auto rs = make_rsrc(p, n > 0 ? (uint32_t)((n < 16 ? n : 16) - 1) * ld2 + 2 * a.dim : 0u);
#pragma unroll
            for (int b = 0; b < C::DB; ++b) lds_dma16<false>(rs, dst + b * C::BN * 64 + rg * 1024, off[b]);
        } else {
            if (keys) k.template copy_lanes<false>(dst, t, rg, next.e, lane);
            else k.template copy_lanes<true>(dst, t, rg, next.e, lane);
        }
    };
    const int kb0 = attn_kbase(lane, 0), kb1 = attn_kbase(lane, 1), vb = attn_vbase(lane);
    if (k.i0 < k.i1) {
        look(k.i0);
        copy(k.i0, 0, std::false_type{});
        if (k.i0 + 1 < k.i1) look(k.i0 + 1);
    }
    // Queries come through LDS as the keys do: 4 lanes bring 64 bytes of a row, where
    // the fragments' own loads would ask for 32 at a time.
    unsigned char* qs = lds + C::QUERIES + wave * C::TILE;
    for (int g = 0; g < 2; ++g) k.copy_queries(qs, wrow + 16 * g + (lane >> 2), g, lane);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");        // (the first tile is waited for too)
#pragma unroll
    for (int j = 0; j < C::KS; ++j) q[j] = *(const u4_t*)(qs + ((j & 1) ? kb1 : kb0) + (j >> 1) * C::BN * 64);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // before the second tile comes here
#pragma unroll
    for (int j = 0; j < C::KS; ++j) asm volatile("" : "+v"(q[j]));
    // INNER: the wave's rows see all of the tile, and the next one is whole.
    int slot = 2 * C::TILE;       // of tile i - 1
    auto step = [&](int i, auto INNER) __attribute__((always_inline)) {
        barrier_vm<0>();          // tile i is in LDS, and everyone is done with tile i - 1
        const int t = k.tile(i), at = t * C::BN, other = slot;
        slot = 2 * C::TILE - slot;
        const unsigned char* kt = lds + slot;
        const unsigned char* vt = kt + C::TILE;
        // Fragments are read ahead of their use, four keys' under the next tile's
        // addresses, the first half of the values' under the softmax: a wave then
        // waits for LDS once a product, not once an instruction.
        auto key = [&](int j) __attribute__((always_inline)) {
            return *(const u4_t*)(kt + ((j & 1) ? kb1 : kb0) + (j >> 1) * C::BN * 64);
        };
        u4_t f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = key(j);
        __builtin_amdgcn_sched_barrier(0);
        if (INNER.value || i + 1 < k.i1) {
            copy(i + 1, other, INNER);
            if (i + 2 < k.i1) look(i + 2);
        }
        if (!INNER.value && (t >= done || (C::WIN && at + C::BN <= dark && at >= a.sinks))) return;
        f16x_t s[1] = {f16x_t{}};
#pragma unroll
        for (int j = 0; j < C::KS; ++j) {
            s[0] = M::mma(f[j & 3], q[j], s[0]);
            if (j + 4 < C::KS) f[j & 3] = key(j + 4);
        }
#pragma unroll
        for (int b = 0; b < C::DB; ++b) f[b] = attn_vfrag<C::BN>(vt, vb, b, 0);
        __builtin_amdgcn_sched_barrier(0);
        if (!INNER.value && (t >= clear || (C::WIN && at < open && at + C::BN > a.sinks)))
            key_mask<C::WIN>(s[0], lim - at, lo - at, a.sinks - 4 * h - at);
        key_move_max<C::DB>(attn_max<1>(s), st, o, a.sc);
        attn_probs<1>(s, st, a.sc);
        u4_t p = attn_pack<C::DT>(s[0], 0);
#pragma unroll
        for (int b = 0; b < C::DB; ++b) {
            o[b] = M::mma(f[b], p, o[b]);
            f[b] = attn_vfrag<C::BN>(vt, vb, b, 1);
        }
        p = attn_pack<C::DT>(s[0], 1);
#pragma unroll
        for (int b = 0; b < C::DB; ++b) o[b] = M::mma(f[b], p, o[b]);
    };
    // The inner tiles need none of the questions that those at the borders ask.
    int in0 = k.i0, in1 = (clear < k.w.nk / C::BN - 1 ? clear : k.w.nk / C::BN - 1) - k.gap;
    if constexpr (C::WIN) {
        const int first = open > 0 ? (open + C::BN - 1) / C::BN - k.gap : 0;
        in0 = first > in0 ? first : in0;
        if (k.gap) in0 = k.sink_tiles > in0 ? k.sink_tiles : in0;
    }
    in1 = in1 < k.i1 - 1 ? in1 : k.i1 - 1;
    int i = k.i0;
    for (const int end = in0 < k.i1 ? in0 : k.i1; i < end; ++i) step(i, std::false_type{});
    for (; i < in1; ++i) step(i, std::true_type{});
    for (; i < k.i1; ++i) step(i, std::false_type{});
    const int lane1 = lane_again(), rr1 = wrow + (lane1 & 31), h1 = lane1 >> 5;
    if (!attn_finite<C>(o, st)) key_again<C>(k, o, st, rr1, k.i0, 1, lane1);
    if (k.w.parts == 1) {
        attn_store<C::DT, C::DB, false>(a, o, st, k.w.q0, k.kvh, rr1, k.rows, 0, lane1);
        return;
    }
    const float l = st.l + other_half(st.l), inv = l == 0.f ? 0.f : 1.f / l;
    if (rr1 >= k.rows) return;
    const int64_t row = k.part_row(rr1);
    if (h1 == 0) a.part_lse[row] = l == 0.f ? -__builtin_inff() : st.m + __builtin_amdgcn_logf(l);
#pragma unroll
    for (int b = 0; b < C::DB; ++b)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int c = 32 * b + 8 * x + 4 * h1;
            if (c < a.dim)
                *(f4_t*)(a.part + row * a.dim + c) =
                    f4_t{o[b][4 * x] * inv, o[b][4 * x + 1] * inv, o[b][4 * x + 2] * inv, o[b][4 * x + 3] * inv};
        }
}

// ---------------------------------------------------------------------------
// Up to 32 rows: the waves take different keys (attn_rows_body's scheme)
// ---------------------------------------------------------------------------
// What bounds it is the bytes of K and V.  Measured (bf16, 32 heads of 128 on 8 key
// heads): 64 requests of up to 8192 keys in pages of 16, 1.02 GB, in 196 us and 5.1
// for the join, 5.05 TB/s in all (a copy of 1 GiB: 5.0 to 5.1); 64 of 8192 each
// 400 to 412 us, 5.2 to 5.4 TB/s; one request of 2048 keys 13 us, of 32768 37 to 42.
// A compute unit holds two workgroups, of which each takes some 7.5 us for a request
// of up to 32 keys: 64 such requests 8.4 us, 128 15.4, 256 31, 512 63.
template <class C>
__device__ __forceinline__ void key_rows_body(const KeyTile<C>& k, unsigned char* lds) {
    using M = Ty32<C::DT>;
    const KeyArgs& a = k.a;
    const int lane = lane_again(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int rr = k.row0 + (lane & 31), h = lane >> 5;
    const int lim = k.sees(rr) - 4 * h, lo = C::WIN ? k.from(rr) - 4 * h : 0;
    const int last = k.rows - 1;
    // tiles below `clear` are seen whole by every row, but for what the window hides of those below `open`
    const int clear = k.sees(k.row0) / C::BN, open = C::WIN ? k.from(last) : 0;
    u4_t q[C::KS];
    f16x_t o[C::DB];
    RowState st;
    attn_load_q<C::KS>(q, a, k.w.q0, k.kvh, rr, k.rows, lane);
    st.init();
#pragma unroll
    for (int b = 0; b < C::DB; ++b) o[b] = f16x_t{};
    unsigned char* mine = lds + wave * C::MINE;
    const int kb0 = attn_kbase(lane, 0), kb1 = attn_kbase(lane, 1), vb = attn_vbase(lane);
    const int i0 = k.i0 + wave;
    auto copy = [&](auto VALUES, unsigned char* dst, int t, int e0, int e1) __attribute__((always_inline)) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");    // what the rows held has been read
        if constexpr (C::PAGED) {
            k.template copy_lanes<VALUES.value>(dst, t, 0, e0, lane);
            k.template copy_lanes<VALUES.value>(dst, t, 1, e1, lane);
        } else {
            k.template copy_packed<VALUES.value>(dst, t, 0, lane);
            k.template copy_packed<VALUES.value>(dst, t, 1, lane);
        }
    };
    f16x_t s[1];
    auto scores = [&]() __attribute__((always_inline)) {
        s[0] = f16x_t{};
#pragma unroll
        for (int j = 0; j < C::KS; ++j)
            s[0] = M::mma(*(const u4_t*)(mine + ((j & 1) ? kb1 : kb0) + (j >> 1) * C::BN * 64), q[j], s[0]);
    };
    u4_t p[2];
    auto softmax = [&](int t) __attribute__((always_inline)) {
        const int at = t * C::BN;
        if (t >= clear || (C::WIN && at < open && at + C::BN > a.sinks))
            key_mask<C::WIN>(s[0], lim - at, lo - at, a.sinks - 4 * h - at);
        key_move_max<C::DB>(attn_max<1>(s), st, o, a.sc);
        attn_probs<1>(s, st, a.sc);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) p[ks] = attn_pack<C::DT>(s[0], ks);
    };
    auto output = [&](const unsigned char* v) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < C::DB; ++b)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) o[b] = M::mma(attn_vfrag<C::BN>(v, vb, b, ks), p[ks], o[b]);
    };
    int e0 = 0, e1 = 0;
    if (i0 < k.i1) {
        e0 = k.entry_of(k.tile(i0), 0, lane);
        e1 = k.entry_of(k.tile(i0), 1, lane);
    }
    if constexpr (C::FEW) {
        // Keys and values have rows of their own: the next tile's keys are under way
        // under the softmax, its values under the next scores, so that a wave waits
        // for one latency a tile and has 8 to 16 KB in flight all the time.  Waits
        // count instructions (2 DB a copy), so nothing else may load in the loop: the
        // table's entries come through LDS too, two tiles ahead.
        unsigned char* values = mine + C::TILE;
        unsigned char* entries = values + C::TILE;
        auto ask = [&](int i) __attribute__((always_inline)) {
            const int key = k.tile(i) * C::BN + (lane & 31);
            lds_dma4_from(entries, a.table + k.w.seq * a.table_ld + a.page(key < k.w.nk ? key : k.w.nk - 1));
        };
        if (i0 < k.i1) {
            if (i0 + C::WAVES < k.i1) ask(i0 + C::WAVES);
            copy(std::false_type{}, mine, k.tile(i0), e0, e1);
            copy(std::true_type{}, values, k.tile(i0), e0, e1);
        }
        for (int i = i0; i < k.i1; i += C::WAVES) {
            const int t = k.tile(i);
            const bool more = i + C::WAVES < k.i1;
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * C::DB) : "memory");         // all but the values
            scores();
            if (more) {
                e0 = ((const int*)entries)[lane >> 2];
                e1 = ((const int*)entries)[16 + (lane >> 2)];
                asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(e0), "+v"(e1)::"memory");
                const int after = i + 2 * C::WAVES < k.i1 ? i + 2 * C::WAVES : i + C::WAVES;
                ask(after);
                copy(std::false_type{}, mine, k.tile(i + C::WAVES), e0, e1);
            }
            softmax(t);
            if (more) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * C::DB + 1) : "memory");     // all but entries and keys
            else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            output(values);
            if (more) copy(std::true_type{}, values, k.tile(i + C::WAVES), e0, e1);
        }
    } else {
        if (i0 < k.i1) copy(std::false_type{}, mine, k.tile(i0), e0, e1);
        for (int i = i0; i < k.i1; i += C::WAVES) {
            const int t = k.tile(i);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            scores();
            copy(std::true_type{}, mine, t, e0, e1);
            int n0 = 0, n1 = 0;
            if (i + C::WAVES < k.i1) {
                n0 = k.entry_of(k.tile(i + C::WAVES), 0, lane);
                n1 = k.entry_of(k.tile(i + C::WAVES), 1, lane);
            }
            softmax(t);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            output(mine);
            e0 = n0;
            e1 = n1;
            if (i + C::WAVES < k.i1) copy(std::false_type{}, mine, k.tile(i + C::WAVES), e0, e1);
        }
    }
    const int lane1 = lane_again(), rr1 = k.row0 + (lane1 & 31);
    if (!attn_finite<C>(o, st)) key_again<C>(k, o, st, rr1, i0, C::WAVES, lane1);
    // join: every wave's maximum and sum, then its rows, scaled to the common maximum
    float* ms = (float*)(lds + C::JOIN);           // [maximum, sum][wave][row]
    const float l = st.l + other_half(st.l);
    if (lane1 < 32) {
        ms[wave * 32 + lane1] = st.m;
        ms[(C::WAVES + wave) * 32 + lane1] = l;
    }
    __syncthreads();
    float m = kLowest, sum = 0.f;
#pragma unroll
    for (int v = 0; v < C::WAVES; ++v) m = __builtin_fmaxf(m, ms[v * 32 + (lane1 & 31)]);
#pragma unroll
    for (int v = 0; v < C::WAVES; ++v)
        sum += ms[(C::WAVES + v) * 32 + (lane1 & 31)] * __builtin_amdgcn_exp2f(ms[v * 32 + (lane1 & 31)] - m);
    const float f = __builtin_amdgcn_exp2f(st.m - m) * (sum == 0.f ? 0.f : 1.f / sum);
    const bool whole = k.w.parts == 1;
    if (wave == 0 && lane1 < 32 && rr1 < k.rows) {
        const float lse2 = sum == 0.f ? -__builtin_inff() : m + __builtin_amdgcn_logf(sum);
        const int pos = a.group(rr1);
        if (!whole) a.part_lse[k.part_row(rr1)] = lse2;
        else if (a.lse) a.lse[(int64_t)(k.w.q0 + pos) * a.heads + k.kvh * a.group.d + (rr1 - pos * a.group.d)] = lse2 * kLn2;
    }
    const int live = k.rows - k.row0;              // 32 at most
    // half of the columns at a time: a wave's tile of LDS holds 32 rows of
    // 16 DB floats, [column quad][row]
    float* mo = (float*)(lds + wave * C::TILE);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        __syncthreads();
#pragma unroll
        for (int x = 0; x < 2 * C::DB; ++x) {
            const int y = half * 2 * C::DB + x, b = y / 4, g = y % 4;        // column quads 2y and 2y + 1
            f4_t v;
            // a wave that weighs nothing here gives its infinities and NaN all the same
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float z = o[b][4 * g + r];
                v[r] = f == 0.f ? (__builtin_fabsf(z) <= -kLowest ? 0.f : z) : z * f;
            }
            *(f4_t*)(mo + ((2 * x + (lane1 >> 5)) * 32 + (lane1 & 31)) * 4) = v;
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
                for (int z = 0; z < 4; ++z) v[z] += y[z];
            }
            const int r = k.row0 + row;
            if (!whole) {
                *(f4_t*)(a.part + k.part_row(r) * a.dim + col) = v;
            } else {
                const int pos = a.group(r), head = k.kvh * a.group.d + (r - pos * a.group.d);
                *(u2_t*)((char*)a.O + ((int64_t)(k.w.q0 + pos) * a.ldo + (int64_t)head * a.hso + col) * 2) =
                    u2_t{Ty<C::DT>::pack(v[0], v[1]), Ty<C::DT>::pack(v[2], v[3])};
            }
        }
    }
}

template <class C>
__global__ __launch_bounds__(C::THREADS, C::PER_CU) void key_attn_kernel(KeyArgs a) {
    __shared__ __attribute__((aligned(1024))) unsigned char lds[C::LDS_BYTES];
    // Workgroups go to the XCDs in turn.  A key head's own row tiles read the same
    // keys: neighbours in `u` with 8 key heads share an XCD's L2.  Few rows a sequence
    // share nothing but the lines on a row's borders, and an XCD should see all heads
    // of a row, which lie on all of its L2's channels (36 requests under a window of
    // 2048, 4 key heads of 96: 34.2 us -> 31.6; rows of prompts would lose their L2:
    // 32768 tokens 1823 us -> 2170, 8001 in 17 sequences 65 -> 74).
    int u, kvh;
    if (a.spread) {
        const int j = (int)blockIdx.x >> 3;
        u = a.kv_heads(j);
        kvh = j - u * a.kv_heads.d;
        u = u * 8 + ((int)blockIdx.x & 7);
    } else {
        u = a.kv_heads((int)blockIdx.x);
        kvh = (int)blockIdx.x - u * a.kv_heads.d;
    }
    KeyItem w;
    if (!C::PAGED && !a.split && a.seqs <= 64) {
        // whole row tiles, those that see the most first (see find_tile_by_size)
        SeqTile x;
        const bool found = a.seqs == 1 ? only_tile(a.cu_q, a.cu_k, (int)a.rows, (int)a.keys, a.group.d, C::BM, u, &x)
                                       : find_tile_by_size(a.cu_q, a.cu_k, a.seqs, (int)a.rows, (int)a.keys, a.group.d, C::BM,
                                                           true, u, &x);
        if (!found) return;
        w = KeyItem{x.seq, x.local, 0, 1, 0, 0, x.q0, x.nq, x.k0, x.nk, x.tiles};
    } else if (!find_item<C::PAGED, C::WIN, false>(a, u, &w)) {
        return;
    }
    const KeyTile<C> k(a, w, kvh);
    if (k.rows - k.row0 <= 32) key_rows_body<C>(k, lds);
    else key_tile_body<C>(k, lds);
}

// ---------------------------------------------------------------------------
// Joining partial results: 32 rows of a tile a workgroup, 16 lanes a row, 8
// columns a lane
// ---------------------------------------------------------------------------
// O = sum_s w_s O_s / sum_s w_s with w_s = 2^(lse_s - max), in one pass with a
// running maximum.  Parts that saw no key have lse = -inf and are left out,
// whatever they hold; infinities and NaN of the others stay, also where the weight
// is 0.  SUB: groups of 16 lanes that a row's parts go over, for few rows.  PER:
// parts whose loads are in flight, 4 for few rows, whose parts are many, 2 for
// tiles, of which more workgroups then fit (276 tiles of 96 columns in two parts
// each: 8.6 us with 2, 10.4 with 4, 15 with 8; 50, 84 and 135 registers).
template <int DT, int PER, int SUB>
__device__ __forceinline__ void key_join_rows(const KeyArgs& a, const KeyItem& w, int kvh, int first, int live, int row0) {
    const int lane = threadIdx.x & 15, sub = SUB == 1 ? 0 : (threadIdx.x >> 4) & (SUB - 1);
    const bool in = 8 * lane < a.dim;
    const int64_t step = (int64_t)w.per_part * a.kv_heads.d * 32;      // from a part's row to the next part's
    for (int r = threadIdx.x / (16 * SUB); r < live; r += 16 / SUB) {
        const int rr = row0 + first + r;
        const int64_t at = ((int64_t)(w.granule + (first >> 5)) * a.kv_heads.d + kvh) * 32 + r;
        float m = -__builtin_inff(), sum = 0.f, x[8] = {};
        auto scale_to = [&](float m1) __attribute__((always_inline)) {
            const float f = __builtin_amdgcn_exp2f(m - (m1 == -__builtin_inff() ? 0.f : m1));
            m = m1;
            sum *= f;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= f;
        };
        for (int s0 = sub; s0 < w.parts; s0 += PER * SUB) {
            float l[PER], m1 = m;
            f4_t v[PER][2];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                l[i] = -__builtin_inff();
                v[i][0] = v[i][1] = f4_t{0.f, 0.f, 0.f, 0.f};
                if (s0 + i * SUB < w.parts) {
                    const int64_t p = at + (s0 + i * SUB) * step;
                    l[i] = a.part_lse[p];
                    if (in) {
                        v[i][0] = *(const f4_t*)(a.part + p * a.dim + 8 * lane);
                        v[i][1] = *(const f4_t*)(a.part + p * a.dim + 8 * lane + 4);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) m1 = __builtin_fmaxf(m1, l[i]);
            scale_to(m1);
            const float m0 = m1 == -__builtin_inff() ? 0.f : m1;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const float f = __builtin_amdgcn_exp2f(l[i] - m0);
                sum += f;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = __builtin_fmaf(f, v[i][e >> 2][e & 3], x[e]);
            }
        }
        if constexpr (SUB > 1) {
            float m1 = m;
#pragma unroll
            for (int d = 16; d < 16 * SUB; d <<= 1) m1 = __builtin_fmaxf(m1, __shfl_xor(m1, d));
            scale_to(m1);
#pragma unroll
            for (int d = 16; d < 16 * SUB; d <<= 1) {
                sum += __shfl_xor(sum, d);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] += __shfl_xor(x[e], d);
            }
        }
        float z = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) z = __builtin_fmaf(x[e], 0.f, z);
        if (__any(z != 0.f)) {
            // infinities or NaN among the parts: a weight of 0, or a rescaling by 0, has made NaN of some
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0.f;
            const float m0 = m == -__builtin_inff() ? 0.f : m;
#pragma unroll 1
            for (int s = 0; s < w.parts; ++s) {
                const int64_t p = at + s * step;
                const float l = a.part_lse[p], f = __builtin_amdgcn_exp2f(l - m0);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float y = in && l != -__builtin_inff() ? a.part[p * a.dim + 8 * lane + e] : 0.f;
                    x[e] += __builtin_fabsf(y) <= -kLowest ? f * y : y;
                }
            }
        }
        if (sub) continue;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int pos = a.group(rr), head = kvh * a.group.d + (rr - pos * a.group.d);
        const int64_t row = w.q0 + pos;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= inv;
        if (in)
            *(u4_t*)((char*)a.O + (row * a.ldo + (int64_t)head * a.hso + 8 * lane) * 2) =
                u4_t{Ty<DT>::pack(x[0], x[1]), Ty<DT>::pack(x[2], x[3]), Ty<DT>::pack(x[4], x[5]), Ty<DT>::pack(x[6], x[7])};
        if (lane == 0 && a.lse)
            a.lse[row * a.heads + head] = sum == 0.f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(sum)) * kLn2;
    }
}

template <int DT, int PER, bool PAGED, bool WIN>
__global__ __launch_bounds__(256) void key_join_kernel(KeyArgs a) {
    const int v = a.kv_heads((int)blockIdx.x), kvh = (int)blockIdx.x - v * a.kv_heads.d;
    KeyItem w;
    const int tile = a.subs == 1 ? v : v >> 2;
    if (!find_item<PAGED, WIN, true>(a, tile, &w) || w.parts == 1) return;
    const int first = a.subs == 1 ? 0 : 32 * (v & 3), row0 = (w.tiles - 1 - w.tile) * kKeyRows;
    int live = w.nq * a.group.d - row0 - first;
    live = live < 32 ? live : 32;
    if (live <= 4) key_join_rows<DT, PER, 4>(a, w, kvh, first, live, row0);
    else if (live <= 8) key_join_rows<DT, PER, 2>(a, w, kvh, first, live, row0);
    else key_join_rows<DT, PER, 1>(a, w, kvh, first, live, row0);
}

}  // namespace b2bk
