// The tiled matrix product of product.h on the matrix units (gfx950).
//
// A workgroup computes a tile of BM x BN results in steps of 128 bytes of k for each row (64
// bfloat16 or 32 float32 values).  A step's tiles of A and B lie in LDS, two steps' in turn:
// while one is multiplied the next is on its way.  A step is two slices of 64 bytes of k, and
// the next slice's fragments are read while a slice is multiplied, also across the step's
// only barrier, so the matrix units wait for neither LDS nor the barrier:
//
//     read slice 1 | multiply slice 0 | next step landed, barrier | start the copy of the step
//     after the next | read the next step's slice 0 | multiply slice 1
//
// Products are computed transposed, (B rows) x (A rows)^T, and the B rows of a wave's matrix
// tiles are interleaved, so that a lane ends with 4 NT consecutive columns of each of its rows
// and stores (and loads the residual) in whole 16-byte pieces.
//
// LDS layouts.  An operand whose k is contiguous: rows of 128 bytes, 16-byte piece q of row r
// at place q ^ key(r).  An operand whose rows are contiguous: lines of one k, BM or BN values,
// 16-byte piece q of line k at place q ^ key(k); bfloat16 fragments are transpose reads
// (ds_read_b64_tr_b16), float32 ones single values.  The keys spread the lanes of one LDS
// cycle over its banks where k is contiguous; transpose reads still meet (cycles of conflicts over
// cycles of accesses in a tile of 256: none, 0.25 with B's rows contiguous, 0.50 with both operands').
//
// Rows and columns past the result's end repeat the last row's or hold what lies beside it:
// they meet no result that is stored.  Values past K are zeros in both operands.
//
// Bound by the matrix units where tiles divide among the CUs, and then by their clock, and by lines
// that come late from behind the L2: 8192^3 in bfloat16 800 us (1375 TFLOP/s, units busy 59 to 66%
// at 1.8 to 2.0 GHz; a step of a 256 tile takes them 2048 cycles of about 2900), 4096^3 in float32
// 930 us (148 TFLOP/s).
#pragma once

#include <type_traits>
#include <utility>

#include "product.h"
#include "ssd_tile.h"

namespace ssd {

constexpr int kStepBytes = 128;

#define SSD_INLINE __attribute__((always_inline))     // of a lambda: its captures stay in registers

constexpr int kAhead = 3;         // the step whose lines are touched, after the one multiplied

constexpr int min_of(int a, int b) { return a < b ? a : b; }

// f(0), f(1), .. f(N - 1) with constants for arguments
template <class F, int... I>
__device__ __forceinline__ void each_index(F f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each_of(F f) {
    each_index(f, std::make_integer_sequence<int, N>{});
}

// One operand's tile of R rows in LDS, and how a wave's fragments take its rows: row i of
// fragment j is 4 NT (i / 4) + 4 j + i % 4 (INTER, NT fragments) or 16 j + i.
template <typename T, int R, bool ROWS_, bool INTER, int NT>
struct TileLayout {
    static constexpr bool ROWS = ROWS_;
    static constexpr int E = (int)sizeof(T), V = 16 / E, KS = kStepBytes / E, SIZE = R;
    static constexpr int BYTES = R * kStepBytes;
    static constexpr int PIECES = ROWS ? R / V : 8;         // 16-byte pieces per LDS line
    static constexpr int PITCH = PIECES * 16;
    // what the places of a line's pieces are XORed with
    __host__ __device__ static constexpr int key(int line) {
        if (!ROWS) return INTER ? (line & 3) | ((line / (4 * NT)) & 1) << 2 : line & 7;
        if (E == 2 && PIECES == 8) return (line >> 1 & 1) << (INTER ? 2 : 1);          // lines of 128 bytes
        if (E == 2) return INTER ? (line & 1) | (line >> 1 & 1) << 3 : (line & 3) << 1;
        if (!INTER) return (line >> 2 & 3) << 2;
        return NT == 4 ? line >> 2 & 3 : (line >> 2 & 1) | (line >> 3 & 1) << 3;
    }
    __host__ __device__ static constexpr int row_of(int j, int i) {
        return INTER ? 4 * NT * (i >> 2) + 4 * j + (i & 3) : 16 * j + i;
    }
    __host__ __device__ static constexpr int at(int line, int piece) { return line * PITCH + (piece ^ key(line)) * 16; }
    // The line and piece of the source that belong at the 16 bytes `slot` of the tile
    __host__ __device__ static constexpr int slot_line(int slot) { return slot / PIECES; }
    __host__ __device__ static constexpr int slot_piece(int slot) { return (slot % PIECES) ^ key(slot / PIECES); }
};

template <typename T> struct Frag;
template <> struct Frag<bf16> { typedef bf16x8 type; };
template <> struct Frag<float> { typedef f32x4 type; };

// Fragment j of slice s of the wave whose first row is r0: lane (i, g) holds row_of(j, i),
// k = 8 g + 0..7 of the slice's 32 (bfloat16) or 4 g + 0..3 of its 16 (float32).
template <class L, typename T>
__device__ __forceinline__ typename Frag<T>::type read_frag(const unsigned char *m, int r0, int j, int s, int lane) {
    const int i = lane & 15, g = lane >> 4;
    if constexpr (!L::ROWS) {
        return *reinterpret_cast<const typename Frag<T>::type *>(m + L::at(r0 + L::row_of(j, i), 4 * s + g));
    } else if constexpr (sizeof(T) == 2) {
        // lane i of 16 reads 4 values of line i / 4 and receives column i of the 4 lines
        const int n = r0 + L::row_of(j, 4 * (i & 3)), line = 32 * s + 8 * g + (i >> 2);
        const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
            (lds_bf16x4_t *)(m + L::at(line, n / 8) + (n & 4) * 2));
        const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
            (lds_bf16x4_t *)(m + L::at(line + 4, n / 8) + (n & 4) * 2));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        const int n = r0 + L::row_of(j, i);
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = *reinterpret_cast<const float *>(m + L::at(16 * s + 4 * g + e, n / 4) + (n & 3) * 4);
        return v;
    }
}

__device__ __forceinline__ f32x4 multiply(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 multiply(f32x4 a, f32x4 b, f32x4 c) { return mma_one(a, b, c); }

// BM x BN results by WM x WN waves.  DMA: operands copied to LDS directly (every piece of 16
// bytes lies on 16 and inside a row), otherwise by way of registers from any address.
template <typename T_, int BM_, int BN_, int WM_, int WN_, bool A_ROWS, bool B_ROWS, bool DMA_, ProductKind KIND_>
struct ProductCfg {
    typedef T_ T;
    static constexpr ProductKind KIND = KIND_;
    static constexpr bool DMA = DMA_;
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NW = WM * WN, THREADS = NW * 64;
    static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
    static constexpr int NT = KIND == kGated ? TN / 2 : TN;       // fragments of one interleaved group
    static constexpr int BCOLS = KIND == kGated ? BN / 2 : BN;    // result columns of a tile
    typedef TileLayout<T, BM, A_ROWS, false, TM> LA;
    typedef TileLayout<T, BN, B_ROWS, true, NT> LB;
    static constexpr int KS = kStepBytes / (int)sizeof(T);
    static constexpr int QA = LA::BYTES / 1024 / NW, QB = LB::BYTES / 1024 / NW;   // copies per wave and step
    static_assert(QA * 1024 * NW == LA::BYTES && QB * 1024 * NW == LB::BYTES, "whole waves of 16-byte pieces");
    static constexpr bool TOUCH = DMA && BM == 256;
    static constexpr int WAVES = BM >= 128 ? 2 : 4;               // of a SIMD at least: registers for its tiles
    static_assert(KIND != kGated || (TN % 2 == 0 && !B_ROWS), "gate and up rows side by side");
};

// Row of B that row r of a tile stands for, from the tile's first column n0, before clamping:
// in a gated product the tile's second half is the other half of B.
template <class C>
__device__ __forceinline__ int64_t b_row(const ProductArgs &p, int64_t n0, int r) {
    if constexpr (C::KIND == kGated)
        return r < C::BN / 2 ? min(n0 + r, p.N - 1) : p.N + min(n0 + r - C::BN / 2, p.N - 1);
    return min(n0 + r, p.N - 1);
}

// What a workgroup does: its tile, its steps of K from `first` on, and, where its tile is shared,
// which of the partial results it leaves (-1: none).
struct Work {
    int m, n;
    int64_t first;
    int steps, part;
};

// Consecutive workgroups go to the 8 XCDs in turn: the i-th of n workgroups in an order in which
// each XCD takes a contiguous range.
__device__ __forceinline__ int xcd_order(int i, int n) {
    const int per = n / 8, more = n % 8, x = i % 8;
    return x * per + min(x, more) + i / 8;
}

__device__ __forceinline__ Work work_of(const ProductGrid &g, int id, int64_t steps) {
    Work w;
    if (id < g.full) {
        id = xcd_order(id, g.full);
        w.first = 0;
        w.steps = (int)steps;
        w.part = -1;
    } else {
        const int i = xcd_order(id - g.full, g.rest * g.splits), split = i / g.rest, tile = i % g.rest;
        id = g.full + tile;
        w.first = (int64_t)split * g.steps;
        w.steps = (int)min((int64_t)g.steps, steps - w.first);
        w.part = tile * g.splits + split;
    }
    const TileAt at = tile_at(id, g);
    w.m = at.m;
    w.n = at.n;
    return w;
}

// The work of workgroup `block` of a product's grid, in LDS of the kernel's.
template <class C>
__device__ __forceinline__ void product_tile(const ProductArgs &p, const Epilogue &ep, const ProductGrid &grid, int block,
                                             unsigned char *A0, unsigned char *B0, unsigned char *A1, unsigned char *B1,
                                             unsigned char *unread) {
    typedef typename C::T T;
    typedef typename Frag<T>::type F;
    typedef typename C::LA LA;
    typedef typename C::LB LB;
    constexpr int E = (int)sizeof(T), V = 16 / E;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / C::WN, wn = w % C::WN;
    const int64_t all = (p.K + C::KS - 1) / C::KS;
    const Work work = work_of(grid, block, all);
    const int64_t m0 = (int64_t)work.m * C::BM, n0 = (int64_t)work.n * C::BCOLS;
    const int steps = work.steps;
    const int64_t k_first = work.first * C::KS;
    const int tail = work.first + steps == all && p.K % C::KS ? steps - 1 : -1;      // the step that K ends in

    // ---- copies
    const int64_t a_size = LA::ROWS ? p.a.size : p.M, b_size = LB::ROWS ? p.b.size : C::KIND == kGated ? 2 * p.N : p.N;
    // 32-bit offsets of this lane's pieces from a scalar base that moves with k.  Copies by way of
    // registers read whole pieces where the operand's rows are contiguous too: one that reaches
    // past the rows reads the next line's first values, and one behind them the tile's first,
    // which meet no result that is stored.
    uint32_t offa[C::QA], offb[C::QB];
    auto offsets = [&](auto layout, const Operand &o, int64_t at, int64_t size, bool is_b, int Q, uint32_t *off) SSD_INLINE {
        typedef decltype(layout) L;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int slot = (w * Q + q) * 64 + lane, line = L::slot_line(slot), piece = L::slot_piece(slot);
            if (L::ROWS) {
                const int64_t n = C::DMA || at + piece * V < size ? at + piece * V : max(min(at, size - V), (int64_t)0);
                off[q] = (uint32_t)((line * o.ld + n - (C::DMA ? at : max(min(at, size - V), (int64_t)0))) * E);
            } else {
                const int64_t r = is_b ? b_row<C>(p, at, line) : min(at + line, size - 1);
                off[q] = (uint32_t)((r - at) * o.ld * E) + piece * 16;
            }
        }
    };
    offsets(LA{}, p.a, m0, a_size, false, C::QA, offa);
    offsets(LB{}, p.b, n0, b_size, true, C::QB, offb);
    u32x4 ra[C::DMA ? 1 : C::QA], rb[C::DMA ? 1 : C::QB];
    // An operand's source: where the next step to copy begins, the bytes from one step to the next,
    // and those that a copy may read from there on, of the split's last step and of others, which
    // reach to the end of the operand's next line.  Copies read zeros past them.
    struct Source {
        const unsigned char *at;
        int64_t step;
        uint32_t whole, last;
    };
    auto source = [&](auto layout, const Operand &o, int64_t row, int64_t size) SSD_INLINE {
        typedef decltype(layout) L;
        auto bytes = [&](int64_t k) SSD_INLINE {
            const int64_t in = (k + V - 1) / V * V;               // lines are whole pieces, zeros past K
            return (uint32_t)min((L::ROWS ? (k - 1) * o.ld + size - row : (size - 1 - row) * o.ld + in) * E, (int64_t)0x7fffffff);
        };
        return Source{reinterpret_cast<const unsigned char *>(o.p) + (L::ROWS ? k_first * o.ld + row : row * o.ld + k_first) * E,
                      (L::ROWS ? o.ld * C::KS : C::KS) * E, bytes(C::KS + 1),
                      bytes(min(p.K - k_first - (int64_t)(steps - 1) * C::KS, (int64_t)C::KS))};
    };
    // Copies `from` to `end` - 1 of step t of an operand; steps are copied in order, and the copies
    // that end one move the source on.  Steps past the split's last read nothing and write zeros
    // that meet no product.
    auto copies = [&](auto layout, Source &src, int t, int from, int end, int Q, const uint32_t *off,
                      unsigned char *to) SSD_INLINE {
        if (from == end) return;
        const rsrc_t rs = make_rsrc(src.at, t + 1 < steps ? src.whole : t < steps ? src.last : 0u);
#pragma unroll
        for (int q = from; q < end; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t *)(to + (w * Q + q) * 1024), 16, off[q], 0, 0, 0);
        if (end == Q) src.at += src.step;
    };
    // Zeros for what a copy of the step that K ends in took from behind K, where the operand's k is
    // contiguous: the rest of its rows, or the next rows.
    auto clear_tail = [&](auto layout, unsigned char *m) SSD_INLINE {
        typedef decltype(layout) L;
        if constexpr (!L::ROWS) {
            const int have = ((int)(p.K % C::KS) + V - 1) / V;
            for (int slot = threadIdx.x; slot < L::BYTES / 16; slot += C::THREADS)
                if (L::slot_piece(slot) >= have) *reinterpret_cast<u32x4 *>(m + slot * 16) = u32x4{0, 0, 0, 0};
        }
    };
    // By way of registers.  Steps of which every piece lies in the operand (to the end of its next
    // line, where its rows are contiguous) are fetched whole from any address; the others value by
    // value.
    auto quick = [&](auto layout, const Operand &o, int64_t size) SSD_INLINE {
        typedef decltype(layout) L;
        if (L::ROWS) return size >= V && o.ld >= V && o.ld <= (int64_t)0x70000000 / E / L::KS;
        return o.ld <= (int64_t)0x70000000 / E / (C::KIND == kGated ? p.N + L::SIZE : L::SIZE);
    };
    const bool quick_a = !C::DMA && quick(LA{}, p.a, a_size), quick_b = !C::DMA && quick(LB{}, p.b, b_size);
    auto fetch = [&](auto layout, const Operand &o, int64_t at, int64_t size, bool is_b, bool quickly, int t, int Q,
                     const uint32_t *off, u32x4 *reg) SSD_INLINE {
        typedef decltype(layout) L;
        const int64_t k = k_first + (int64_t)t * C::KS;
        const T *const src = reinterpret_cast<const T *>(o.p);
        if (quickly && (L::ROWS ? work.first + t + 1 < all : t != tail)) {
            const unsigned char *base = reinterpret_cast<const unsigned char *>(
                L::ROWS ? src + k * o.ld + min(at, size - V) : src + at * o.ld + k);
#pragma unroll
            for (int q = 0; q < Q; ++q) __builtin_memcpy(&reg[q], base + off[q], 16);
            return;
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int slot = (w * Q + q) * 64 + lane, line = L::slot_line(slot), piece = L::slot_piece(slot);
            const T *from;
            int64_t have;
            if (L::ROWS) {
                have = k + line < p.K ? size - (at + piece * V) : 0;
                from = src + (k + line) * o.ld + at + piece * V;
            } else {
                const int64_t r = is_b ? b_row<C>(p, at, line) : min(at + line, size - 1);
                have = p.K - (k + piece * V);
                from = src + r * o.ld + k + piece * V;
            }
            T v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = i < have ? from[i] : from_f32<T>(0.f);
            __builtin_memcpy(&reg[q], v, 16);
        }
    };
    auto place = [&](int Q, const u32x4 *reg, unsigned char *to) SSD_INLINE {
#pragma unroll
        for (int q = 0; q < Q; ++q) *reinterpret_cast<u32x4 *>(to + ((w * Q + q) * 64 + lane) * 16) = reg[q];
    };
    Source src_a = source(LA{}, p.a, m0, a_size), src_b = source(LB{}, p.b, n0, b_size);
    auto copies_a = [&](int t, int from, int end, unsigned char *to) SSD_INLINE {
        copies(LA{}, src_a, t, from, end, C::QA, offa, to);
    };
    auto copies_b = [&](int t, int from, int end, unsigned char *to) SSD_INLINE {
        copies(LB{}, src_b, t, from, end, C::QB, offb, to);
    };
    // A line of memory that no workgroup of the XCD has read yet comes from behind its L2, later than a
    // step takes: with every line already there the copies alone of 8192^3 take 0.85 million
    // cycles, as they are 1.67 (the products 1.05).  So the lines of a later step are touched
    // ahead, one access of 4 bytes each, by one of the workgroups that share them: of the 4 tiles of
    // a row each takes a quarter of A's lines, of the 8 of a column an eighth of B's; even waves
    // A's, odd waves B's.  (8192^3: 840 -> 824 us, 783 -> 775 by x, 807 -> 782 by the weight; in
    // the smaller tiles, whose workgroups share a CU, it was not tried.)
    const bool of_b = w & 1;
    Source src_ahead = of_b ? src_b : src_a;
    uint32_t off_ahead = 0x80000000u;                            // none: past every source
    if constexpr (C::TOUCH) {
        static_assert(LA::BYTES == 256 * 128 && LB::BYTES == 256 * 128, "256 lines of 128 bytes a step");
        constexpr int NA = 256 / 4 / (C::NW / 2), NB = 256 / 8 / (C::NW / 2);            // of them a wave's
        const int n = of_b ? NB : NA, line = ((of_b ? work.m % 8 : work.n % 4) * (C::NW / 2) + w / 2) * n + lane;
        if (lane < n) {
            if (of_b ? LB::ROWS : LA::ROWS) {
                off_ahead = (uint32_t)(line / 4 * (of_b ? p.b.ld : p.a.ld) * E) + line % 4 * 128;
            } else {
                const int64_t r = of_b ? b_row<C>(p, n0, line) - n0 : min(m0 + line, p.M - 1) - m0;
                off_ahead = (uint32_t)(r * (of_b ? p.b.ld : p.a.ld) * E);
            }
        }
        src_ahead.at += (kAhead - 1) * src_ahead.step;
    }
    auto touch = [&](int t) SSD_INLINE {
        const rsrc_t rs = make_rsrc(src_ahead.at, t + 1 < steps ? src_ahead.whole : 0u);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t *)(unread + w * 256), 4, off_ahead, 0, 0, 0);
        src_ahead.at += src_ahead.step;
    };
    auto fetch_both = [&](int t) SSD_INLINE {
        fetch(LA{}, p.a, m0, a_size, false, quick_a, t, C::QA, offa, ra);
        fetch(LB{}, p.b, n0, b_size, true, quick_b, t, C::QB, offb, rb);
    };
    // By way of registers: what was fetched (step t) goes to (a, b), and the step after it is
    // fetched.
    auto store_fetch = [&](int t, unsigned char *a, unsigned char *b) SSD_INLINE {
        place(C::QA, ra, a);
        place(C::QB, rb, b);
        if (t + 1 < steps) fetch_both(t + 1);
    };

    // ---- products
    f32x4 acc[C::TM][C::TN];
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
        for (int j = 0; j < C::TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    F a[2][C::TM], b[2][C::TN];
    auto read_b = [&](int s, int j, const unsigned char *m) SSD_INLINE {
        b[s][j] = read_frag<LB, T>(m, (j / C::NT) * (C::BN / 2) + wn * 16 * C::NT, j % C::NT, s, lane);
    };
    auto read_a = [&](int s, int i, const unsigned char *m) SSD_INLINE { a[s][i] = read_frag<LA, T>(m, wm * 16 * C::TM, i, s, lane); };
    auto read = [&](int s, const unsigned char *ma, const unsigned char *mb) SSD_INLINE {
#pragma unroll
        for (int j = 0; j < C::TN; ++j) read_b(s, j, mb);
#pragma unroll
        for (int i = 0; i < C::TM; ++i) read_a(s, i, ma);
    };
    // The products of slice s, one row of tiles after the other, in a fixed order with the reads of
    // the other slice's fragments from (ma, mb), B's first, and the copies that `between` starts.
    // The compiler's own order reads late and waits; a row's fragment is read no earlier than its
    // place in the registers comes free, which keeps 256 registers enough for 8 x 4 tiles.
    auto products = [&](int s, const unsigned char *ma, const unsigned char *mb, auto between) SSD_INLINE {
        constexpr int R = C::TM + C::TN, GROUPS = C::TM > 2 ? C::TM - 1 : C::TM;
        each_of<C::TM>([&](auto at) SSD_INLINE {
            constexpr int i = decltype(at)::value;
            between(at);
            constexpr int first = min_of(R, (i * R + GROUPS - 1) / GROUPS), end = min_of(R, ((i + 1) * R + GROUPS - 1) / GROUPS);
            each_of<end - first>([&](auto r) SSD_INLINE {
                constexpr int q = first + decltype(r)::value;
                if constexpr (q < C::TN) read_b(1 - s, q, mb);
                else read_a(1 - s, q - C::TN, ma);
            });
#pragma unroll
            for (int j = 0; j < C::TN; ++j) acc[i][j] = multiply(b[s][j], a[s][i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // This wave's copies have landed and its LDS reads are done, then every wave's; the compiler
    // moves no access of memory across it.
    auto landed = [&]() SSD_INLINE {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(C::TOUCH ? 0x0071 : 0);        // the last touch, behind the copies, may be on its way
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    auto clear = [&](unsigned char *a, unsigned char *b) SSD_INLINE {
        clear_tail(LA{}, a);
        clear_tail(LB{}, b);
        landed();
    };
    // Step t from (a0, b0); (a1, b1) are the next step's tiles.  The copies start as soon as a0 and b0
    // are free, spread over half a slice (a copy of 64 x 16 bytes takes the memory pipe 16 cycles,
    // and blocks the wave while the pipe is full).  After the last step the fragments read are
    // whatever lies in LDS, and meet no product.
    auto step = [&](int t, unsigned char *a0, unsigned char *b0, unsigned char *a1, unsigned char *b1) SSD_INLINE {
        products(0, a0, b0, [](auto) {});
        landed();
        if constexpr (C::DMA) {
            if (t + 1 == tail) clear(a1, b1);
            products(1, a1, b1, [&](auto at) SSD_INLINE {
                constexpr int i = decltype(at)::value, PARTS = C::TM > 4 ? C::TM / 4 : 1;
                if constexpr (i < PARTS) copies_a(t + 2, i * C::QA / PARTS, (i + 1) * C::QA / PARTS, a0);
                else if constexpr (i < 2 * PARTS)
                    copies_b(t + 2, (i - PARTS) * C::QB / PARTS, (i - PARTS + 1) * C::QB / PARTS, b0);
                else if constexpr (C::TOUCH && i == 2 * PARTS) touch(t + kAhead);
            });
        } else {
            if (t + 2 < steps) store_fetch(t + 2, a0, b0);
            products(1, a1, b1, [](auto) {});
        }
    };
    if constexpr (C::DMA) {
        copies_a(0, 0, C::QA, A0);
        copies_b(0, 0, C::QB, B0);
        __builtin_amdgcn_s_waitcnt(0);
        landed();
        copies_a(1, 0, C::QA, A1);
        copies_b(1, 0, C::QB, B1);
        if constexpr (C::TOUCH) {
            __builtin_amdgcn_sched_barrier(0);                   // behind the copies, which the waits count on
            touch(kAhead - 1);
        }
        if (tail == 0) clear(A0, B0);
    } else {
        fetch_both(0);
        store_fetch(0, A0, B0);
        if (steps > 1) store_fetch(1, A1, B1);
        landed();
    }
    read(0, A0, B0);
    for (int t = 0;;) {
        step(t, A0, B0, A1, B1);
        if (++t >= steps) break;
        step(t, A1, B1, A0, B0);
        if (++t >= steps) break;
    }
    if constexpr (C::DMA) __builtin_amdgcn_s_waitcnt(0x0f70);      // no copy is left behind

    // ---- results: this lane's columns are n .. n + 4 NT - 1 of each half
    const int i16 = lane & 15, g = lane >> 4, col = wn * 16 * C::NT + 4 * C::NT * g;
    if (work.part >= 0) {
        float *part = p.part + (int64_t)work.part * C::BM * C::BN;
#pragma unroll
        for (int i = 0; i < C::TM; ++i) {
            float *row = part + (wm * 16 * C::TM + 16 * i + i16) * C::BN + col;
#pragma unroll
            for (int j = 0; j < C::TN; ++j)
                *reinterpret_cast<f32x4 *>(row + (j / C::NT) * (C::BN / 2) + 4 * (j % C::NT)) = acc[i][j];
        }
        return;
    }
    // what the epilogue reads, all of it before the first store, which the compiler would not pass
    constexpr int W = V < 4 * C::NT ? V : 4 * C::NT, PARTS = 4 * C::NT / W;
    const int64_t n = n0 + col, m = m0 + wm * 16 * C::TM + i16;
    float bias[C::KIND == kGated ? 2 : 1][PARTS][W];
    typename Pack<T, W>::type residual[C::TM][PARTS];
#pragma unroll
    for (int c = 0; c < PARTS; ++c) {
        if constexpr (C::KIND != kPlain) load_bias<T, W>(ep, n + c * W, false, bias[0][c]);
        if constexpr (C::KIND == kGated) load_bias<T, W>(ep, n + c * W, true, bias[1][c]);
        if constexpr (C::KIND == kLinear)
#pragma unroll
            for (int i = 0; i < C::TM; ++i) residual[i][c] = load_residual<T, W>(ep, m + 16 * i, n + c * W);
    }
#pragma unroll
    for (int i = 0; i < C::TM; ++i) {
        if (m + 16 * i >= p.M) break;
#pragma unroll
        for (int c = 0; c < PARTS; ++c) {
            float v[W];
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = acc[i][(c * W + e) / 4][e % 4];
            if constexpr (C::KIND == kGated) {
                float u[W];
#pragma unroll
                for (int e = 0; e < W; ++e) u[e] = acc[i][C::NT + (c * W + e) / 4][e % 4];
                finish_gated<T, W>(ep, m + 16 * i, n + c * W, bias[0][c], bias[1][c], v, u);
            } else if constexpr (C::KIND == kLinear) {
                finish_linear<T, W>(ep, m + 16 * i, n + c * W, bias[0][c], residual[i][c], v);
            } else {
                const int left = (int)min(p.N - (n + c * W), (int64_t)W);
                store_some<T, W>(reinterpret_cast<T *>(ep.y) + (m + 16 * i) * ep.N + n + c * W, left, v);
            }
        }
    }
}

template <class C>
__global__ __launch_bounds__(C::THREADS, C::WAVES) void product_kernel(ProductArgs p, Epilogue ep, ProductGrid grid) {
    __shared__ __align__(16) unsigned char A0[C::LA::BYTES], B0[C::LB::BYTES], A1[C::LA::BYTES], B1[C::LB::BYTES];
    __shared__ __align__(16) unsigned char unread[C::TOUCH ? C::NW * 256 : 16];      // what touched lines leave
    product_tile<C>(p, ep, grid, blockIdx.x, A0, B0, A1, B1, unread);
}

// Two products whose tiles lie in LDS alike: the first's workgroups, then the second's.
template <class C, class D>
__global__ __launch_bounds__(C::THREADS, C::WAVES) void product_pair_kernel(ProductArgs p, Epilogue pe, ProductGrid pg,
                                                                           ProductArgs q, Epilogue qe, ProductGrid qg) {
    static_assert(C::LA::BYTES == D::LA::BYTES && C::LB::BYTES == D::LB::BYTES && C::THREADS == D::THREADS && !C::TOUCH &&
                  !D::TOUCH, "tiles alike");
    __shared__ __align__(16) unsigned char A0[C::LA::BYTES], B0[C::LB::BYTES], A1[C::LA::BYTES], B1[C::LB::BYTES];
    if ((int)blockIdx.x < pg.full) product_tile<C>(p, pe, pg, blockIdx.x, A0, B0, A1, B1, nullptr);
    else product_tile<D>(q, qe, qg, blockIdx.x - pg.full, A0, B0, A1, B1, nullptr);
}

template <class C>
hipError_t launch_tiles(const ProductArgs &a, const ProductGrid &g, hipStream_t s) {
    product_kernel<C><<<(uint32_t)(g.full + g.rest * g.splits), C::THREADS, 0, s>>>(a, epilogue_of(a), g);
    return hipGetLastError();
}

// The launch of one shape of tile for each form of product that there is: k contiguous in both
// operands (linear, gated), the rows contiguous in B (a gradient by x), in both (by a weight).
template <typename T, int BM, int BN, int WM, int WN, bool DMA>
hipError_t launch_tiles_of(const ProductArgs &a, const ProductGrid &g, hipStream_t s) {
    if (a.kind == kGated) return launch_tiles<ProductCfg<T, BM, BN, WM, WN, false, false, DMA, kGated>>(a, g, s);
    if (a.kind == kLinear) return launch_tiles<ProductCfg<T, BM, BN, WM, WN, false, false, DMA, kLinear>>(a, g, s);
    if (a.a_rows) return launch_tiles<ProductCfg<T, BM, BN, WM, WN, true, true, DMA, kPlain>>(a, g, s);
    return launch_tiles<ProductCfg<T, BM, BN, WM, WN, false, true, DMA, kPlain>>(a, g, s);
}

// The launch of both gradients' products, by x and by a weight, in tiles of 64; whole tiles only.
template <typename T>
hipError_t launch_pair_of(const ProductArgs &x, const ProductGrid &gx, const ProductArgs &w, const ProductGrid &gw,
                          bool x_first, hipStream_t s) {
    typedef ProductCfg<T, 64, 64, 2, 2, false, true, true, kPlain> X;
    typedef ProductCfg<T, 64, 64, 2, 2, true, true, true, kPlain> W;
    const uint32_t n = (uint32_t)(gx.full + gw.full);
    if (x_first) product_pair_kernel<X, W><<<n, X::THREADS, 0, s>>>(x, epilogue_of(x), gx, w, epilogue_of(w), gw);
    else product_pair_kernel<W, X><<<n, X::THREADS, 0, s>>>(w, epilogue_of(w), gw, x, epilogue_of(x), gx);
    return hipGetLastError();
}

}  // namespace ssd
