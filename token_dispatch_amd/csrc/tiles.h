// One output tile of a matrix product on the matrix units of gfx950, for the
// experts' products (experts.hip). Not part of the ABI.
//
// D[m][n] = sum_k X[m][k] W[n][k]. A workgroup holds the tile's sums in registers
// and walks k in steps of KB = 128 or 64 bytes of a row: both operands' parts of a step are
// loaded straight into a ring in shared memory (16 bytes a lane, no registers on the
// way), ahead of the step the matrix units work on, with one barrier for each step.
//
// An operand lies in memory in one of two ways:
//   rows   k runs along its rows: the step's part is [BT][KB bytes]
//   cols   k runs across its rows: the step's part is [KB / EB rows of k][BT elements],
//          and lanes get their k values with transposing reads (2-byte elements) or one
//          by one (4-byte elements)
// The 16-byte chunks of a part's rows are exchanged by an XOR with some of the row's
// bits, so that lanes which read the same chunk of different rows hit different banks.
// Loads past the operand's end (rows behind a segment, the last step's k, columns behind
// the matrix) return zeros by the buffer's range check, or land in sums that are not
// stored.
//
// What bounds it, measured at 262144 rows in 64 segments, 2048 -> 1024 columns, tiles of 256 x
// 256: the matrix units are busy for 59% of 0.95 ms (bf16; the clock is at 2.0 GHz then, of 2.4),
// 6% of shared memory's cycles are bank conflicts (those of the epilogue), and the
// loads alone take 0.84 to 0.95 ms: 64 KB a step for each compute unit, a fifth of it
// past the L2, with about as much in flight as the ring holds. So the tile is as large as
// the registers allow (fewer bytes a product), and steps are whole 128-byte lines of each row.
// Smaller tiles with two workgroups on a unit (128 x 256: 1.06 to 1.19 ms), four waves of 128
// x 128 (1.03 to 1.06), more but shorter steps (1.04) and loads that only bring lines to the
// L2 early (0.99 against 1.02 then) were slower or no gain.
#pragma once

#include <type_traits>
#include <utility>

#include "experts.h"
#include "rows.h"

namespace moonep {
namespace tiles {

using namespace rows;

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kOutOfRange = 0x7ffffff0;

__device__ __forceinline__ uint32_t lds_offset(const void *p) {
    return (uint32_t)(uintptr_t)(const lds_char *)p;
}

// 64 lanes x 16 bytes from the buffer at voff into shared memory at `to` + OFFSET onwards,
// lane after lane. Done when vmcnt says so.
template <int OFFSET>
__device__ __forceinline__ void load_to_lds(uint32_t to, int voff, __amdgpu_buffer_rsrc_t rs) {
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"{m0}"(to + OFFSET), "v"(voff), "s"(rs)
                 : "memory");
}

template <typename F, int... I>
__device__ __forceinline__ void each_of(F &&f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>()), ...);
}

// f(0) .. f(N - 1), each with its number as a constant.
template <int N, typename F>
__device__ __forceinline__ void each(F &&f) {
    each_of(f, std::make_integer_sequence<int, N>());
}

__device__ __forceinline__ int wave_id() {
    return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
}

// What lanes of this wave wrote to shared memory before is there for its other lanes after: a
// wave's accesses to shared memory are done in their order, so this only holds the compiler.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const char *p, int records) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), (short)0, records, kWordFormat);
}

// 16 bytes of k for each lane, as the matrix units take them, and their products.
template <int EB>
struct Unit;
template <>
struct Unit<2> {
    typedef v8bf Frag;
    typedef v4f Acc;
    __device__ static Acc mma(Frag a, Frag b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Unit<1> {
    typedef v4i Frag;
    typedef v4i Acc;
    __device__ static Acc mma(Frag a, Frag b, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
    }
};
template <>
struct Unit<4> {
    typedef v4f Frag;
    typedef v4f Acc;
    __device__ static Acc mma(Frag a, Frag b, Acc c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
        return c;
    }
};

// One operand: EB bytes an element, BT rows (of the product's m or n) in a tile, NW waves.
template <int EB, bool COLS, int BT, int NW, int KB>
struct Side {
    static constexpr int kBytes = BT * KB;             // of one step's part
    static constexpr int kLoads = kBytes / 1024 / NW;  // by each wave
    static constexpr int kK = KB / EB;                 // k of one step
    static constexpr int kRow = COLS ? BT * EB : KB;
    static constexpr int kChunks = kRow / 16;
    static_assert(kBytes % (1024 * NW) == 0, "each wave loads whole kilobytes");

    __device__ static int wave() { return NW == 1 ? 0 : wave_id(); }

    // Rows that lanes read at the same chunk, 16 of them for rows and for the transposing
    // reads of cols (four rows each of four k groups), must differ here or in the bank that
    // they begin at.
    __device__ static int swizzle(int row) {
        int v;
        if constexpr (!COLS) v = KB == 128 ? row >> 1 : row >> 2;
        else if constexpr (EB == 4) v = ((row >> 2) & 3) << 2;
        else if constexpr (kChunks >= 16) v = ((row & 3) | ((row >> 3) & 1) << 2) << 1;
        else if constexpr (kChunks == 8) v = (((row >> 1) & 1) | ((row >> 3) & 1) << 1) << 1;
        else v = ((row >> 3) & 1) << 1;
        return v & (kChunks - 1 < 7 || COLS ? kChunks - 1 : 7);
    }

    const char *base;  // first element of the tile
    int ld, left;      // bytes of a row; rows: bytes from base to the operand's end,
                       // cols: bytes of a row before base
    int k;             // cols: rows of k
    // A wave's loads differ in the row alone, or (odd NW) every other one in the chunk too.
    static constexpr int kShapes = !COLS && KB == 128 && NW % 2 == 1 ? 2 : 1;
    int voff[kLoads], chunk[kShapes];

    // p: the operand's tile. rows: `valid` rows follow. cols: k rows, `before` bytes of
    // each lie before the tile.
    __device__ void init(const char *p, int row_bytes, int valid_or_k, int before) {
        base = p;
        ld = row_bytes;
        left = COLS ? before : valid_or_k * row_bytes;
        k = COLS ? valid_or_k : 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = (i * NW + wave()) * 64 + lane_id();
            const int row = at / kChunks, c = (at % kChunks) ^ swizzle(row);
            voff[i] = row * ld + c * 16;
            if (i < kShapes) chunk[i] = c * 16;
        }
    }

    // The loads of step `step`: all of them, or one by one after step().
    __amdgpu_buffer_rsrc_t range;
    int rem;  // rows: bytes of a row from the step on

    __device__ void step(int step) {
        if constexpr (COLS) {
            const int rows = min(k - step * kK, kK);
            range = rsrc(base + (int64_t)step * kK * ld, rows > 0 ? rows * ld - left : 0);
        } else {
            const int at = step * KB;
            rem = ld - at;
            range = rsrc(base + at, max(left - at, 0));
        }
    }

    template <int I>
    __device__ void load_one(uint32_t to) {
        int at = voff[I];
        if constexpr (!COLS) at = chunk[I % kShapes] < rem ? at : kOutOfRange;
        load_to_lds<I * NW * 1024>(to + wave() * 1024, at, range);
    }

    __device__ void load(int s, uint32_t to) {
        step(s);
        each<kLoads>([&](auto i) { load_one<decltype(i)::value>(to); });
    }

    // The fragment of 16 rows from row `first` on, half `h` of the step.
    typedef typename Unit<EB>::Frag Frag;
    __device__ static Frag read(const char *part, int first, int h) {
        const int l = lane_id(), i = l & 15, g = l >> 4;
        if constexpr (!COLS) {
            return *reinterpret_cast<const Frag *>(part + (first + i) * kRow +
                                                   (((h * 4 + g) ^ swizzle(i)) * 16));
        } else if constexpr (EB == 2) {
            const int row = g * 8 + (i >> 2), c = first / 8 + ((i >> 1) & 1);
            const char *p = part + (h * 32 + row) * kRow + (c ^ swizzle(row)) * 16 + (i & 1) * 8;
            typedef __attribute__((address_space(3))) v4s lds_v4s;
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)p);
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(p + 4 * kRow));
            return __builtin_bit_cast(Frag, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const int row = g * 4, c = first / 4 + (i >> 2);
            const char *p = part + (h * 16 + row) * kRow + (c ^ swizzle(row)) * 16 + (i & 3) * 4;
            Frag f;
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = *reinterpret_cast<const float *>(p + j * kRow);
            return f;
        }
    }
};

// The tile's sums. Wave w of WM x WN holds rows (w / WN) * TM .. and columns
// (w % WN) * TN .., so that with WN = 4 each SIMD has a wave of every row group, and waves
// whose rows are all behind the segment's end leave their SIMD to the others. Lane l of
// acc[n][m] holds row m * 16 + l % 16 and the four columns from n * 16 + l / 16 * 4 on: the
// columns go into the matrix unit's first operand, so that a lane's four sums lie side by
// side in an output row.
//
// With WK > 1 every wave makes the whole tile over every WK-th step, in shared memory of
// its own and without barriers; the waves' sums are added in the waves' order at the end,
// and wave 0 holds the tile.
template <int EB, bool XCOLS, bool WCOLS, int BM, int BN, int WM, int WN, int WK, int STAGES,
          int KB = 128, bool PIPED = false>
struct Product {
    static_assert(WK == 1 || WM * WN == 1, "waves share a tile or the steps");
    static constexpr int kThreads = WM * WN * WK * 64;
    static constexpr int TM = BM / WM, TN = BN / WN;
    typedef Side<EB, XCOLS, BM, WM * WN, KB> X;
    typedef Side<EB, WCOLS, BN, WM * WN, KB> W;
    static constexpr int kStage = X::kBytes + W::kBytes;
    // Shared memory of the waves of one tile: STAGES stages, of half a stage each if PIPED.
    static constexpr int kRing = PIPED ? STAGES * kStage / 2 : STAGES * kStage;
    static constexpr int kLds = WK * kRing;
    static constexpr int kLoads = X::kLoads + W::kLoads;
    typedef typename Unit<EB>::Acc Acc;
    typedef Acc Sums[TN / 16][TM / 16];

    __device__ static int row0() { return WK > 1 ? 0 : wave_id() / WN * TM; }
    __device__ static int col0() { return WK > 1 ? 0 : wave_id() % WN * TN; }
    __device__ static bool holds() { return WK == 1 || wave_id() == 0; }

    // At most N loads in flight, and what the tile's waves loaded is there for all of them.
    template <int N>
    __device__ static void wait() {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
        if constexpr (WK == 1) __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }

    // f[CUR] is multiplied while f[1 - CUR] is read from half `h` of a step's parts; with
    // LOADS the loads that step() has set up go to to_x and to_w. A matrix instruction keeps
    // its unit busy for four issue slots, so the reads and loads go between the products one
    // at a time.
    template <int CUR, bool LOADS, typename F>
    __device__ static void phase(F &f, const char *px, const char *pw, int h, X &x, W &w,
                                 uint32_t to_x, uint32_t to_w, Sums &acc) {
        constexpr int NM = TM / 16, NN = TN / 16, NF = NM + NN, kAll = NM * NN;
        each<kAll>([&](auto at) {
            constexpr int i = decltype(at)::value;
            constexpr int r = i * NF / kAll, l = i * kLoads / kAll;
            if constexpr (r < (i + 1) * NF / kAll)
                f[1 - CUR][r] = r < NN ? W::read(pw, col0() + r * 16, h)
                                       : X::read(px, row0() + (r - NN) * 16, h);
            if constexpr (LOADS && l < (i + 1) * kLoads / kAll) {
                // in the order of the parts, so that the older part is the first to be there
                constexpr bool kX = (l < kLoads / 2) == (STAGES % 2 == 0);
                if constexpr (kX) x.template load_one<l % X::kLoads>(to_x);
                else w.template load_one<l % X::kLoads>(to_w);
            }
            constexpr int n = i / NM, m = i % NM;
            acc[n][m] = Unit<EB>::mma(f[CUR][n], f[CUR][NN + m], acc[n][m]);
            __builtin_amdgcn_sched_barrier(0);
        });
    }

    // Fragments are read a half step ahead of their products, and the barrier stands where a
    // step's last fragments are in registers: its two parts are free then. The ring holds
    // STAGES half stages, X and W parts in turn, so that the loads of a part can be in flight
    // across a barrier where only two whole stages would fit: five parts instead of four took
    // 1.02 to 0.95 ms at the shape above. Operands in cols lose nothing by steps of 64 bytes
    // (their rows are the tile's width), and eight such parts are 3% faster than five of 128.
    __device__ static void run_piped(X &x, W &w, int k, bool busy, char *lds, Sums &acc) {
        constexpr int NM = TM / 16, NN = TN / 16, NF = NM + NN;
        constexpr int kPart = X::kBytes, kAhead = (STAGES - 4) * X::kLoads;
        static_assert(X::kBytes == W::kBytes && STAGES >= 4, "parts of one size, two stages at least");
        const int steps = (k + X::kK - 1) / X::kK;
        const uint32_t base = lds_offset(lds);
        typename X::Frag f[2][NF];
        each<STAGES>([&](auto at) {
            constexpr int p = decltype(at)::value;
            if constexpr (p % 2 == 0) x.load(p / 2, base + p * kPart);
            else w.load(p / 2, base + p * kPart);
        });
        wait<(STAGES - 2) * X::kLoads>();
        if (!busy) {  // loads and waits alone
            uint32_t to_x = base, to_w = base + kPart;
            const int turns = KB == 128 ? steps : (steps + 1) / 2 * 2;
            for (int s = 0; s < turns; ++s) {
                wait<kAhead>();
                if constexpr (STAGES % 2 == 0) {
                    x.load(s + STAGES / 2, to_x);
                    w.load(s + STAGES / 2, to_w);
                } else {
                    w.load(s + STAGES / 2, to_x);
                    x.load(s + STAGES / 2 + 1, to_w);
                }
                to_x += 2 * kPart;
                to_w += 2 * kPart;
                if (to_x >= base + STAGES * kPart) to_x -= STAGES * kPart;
                if (to_w >= base + STAGES * kPart) to_w -= STAGES * kPart;
            }
            wait<0>();
            return;
        }
#pragma unroll
        for (int i = 0; i < NF; ++i)
            f[0][i] = i < NN ? W::read(lds + kPart, col0() + i * 16, 0)
                             : X::read(lds, row0() + (i - NN) * 16, 0);
        int at_x = 0, at_w = kPart;  // the step's parts
        auto turn = [&](int s, auto cur) {
            wait<kAhead>();
            const uint32_t first = base + at_x, second = base + at_w;
            at_x += 2 * kPart;
            at_w += 2 * kPart;
            if (at_x >= STAGES * kPart) at_x -= STAGES * kPart;
            if (at_w >= STAGES * kPart) at_w -= STAGES * kPart;
            // an odd ring is a W part ahead, so the free parts change their kinds
            constexpr bool kOdd = STAGES % 2 == 1;
            x.step(s + (STAGES + 1) / 2);
            w.step(s + STAGES / 2);
            phase<decltype(cur)::value, true>(f, lds + at_x, lds + at_w, 0, x, w, kOdd ? second : first,
                                              kOdd ? first : second, acc);
        };
        typedef std::integral_constant<int, 0> Even;
        typedef std::integral_constant<int, 1> Odd;
        if constexpr (KB == 128) {
            for (int s = 0; s < steps; ++s) {
                phase<0, false>(f, lds + at_x, lds + at_w, 1, x, w, 0, 0, acc);
                turn(s, Odd());
            }
        } else {
            // in pairs: a step past the last one multiplies zeros
            for (int s = 0; s < steps; s += 2) {
                turn(s, Even());
                turn(s + 1, Odd());
            }
        }
        wait<0>();
    }

    // rows: rows of the tile that count (the others' sums may be left out).
    __device__ static void run(X &x, W &w, int k, int rows, char *lds, Sums &acc) {
        const bool busy = row0() < rows;
        const int first = WK > 1 ? wave_id() : 0;
        const int steps = (k + X::kK - 1) / X::kK;
        lds += first * kRing;
        const uint32_t base = lds_offset(lds);
#pragma unroll
        for (int n = 0; n < TN / 16; ++n)
#pragma unroll
            for (int m = 0; m < TM / 16; ++m) acc[n][m] = Acc{0, 0, 0, 0};
        if constexpr (PIPED) {
            run_piped(x, w, k, busy, lds, acc);
            return;
        }
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) {
            x.load(first + s * WK, base + s * kStage);
            w.load(first + s * WK, base + s * kStage + X::kBytes);
        }
        int at = 0, next = (STAGES - 1) * kStage;
        for (int s = first; s < steps; s += WK) {
            wait<(STAGES - 2) * kLoads>();
            // steps past the last one load nothing: their range is empty
            x.load(s + (STAGES - 1) * WK, base + next);
            w.load(s + (STAGES - 1) * WK, base + next + X::kBytes);
            const char *part = lds + at;
            if (busy) {
#pragma unroll
                for (int h = 0; h < KB / 64; ++h) {
                    typename X::Frag fx[TM / 16], fw[TN / 16];
#pragma unroll
                    for (int n = 0; n < TN / 16; ++n)
                        fw[n] = W::read(part + X::kBytes, col0() + n * 16, h);
#pragma unroll
                    for (int m = 0; m < TM / 16; ++m) fx[m] = X::read(part, row0() + m * 16, h);
#pragma unroll
                    for (int n = 0; n < TN / 16; ++n)
#pragma unroll
                        for (int m = 0; m < TM / 16; ++m)
                            acc[n][m] = Unit<EB>::mma(fw[n], fx[m], acc[n][m]);
                }
            }
            at = at + kStage == kRing ? 0 : at + kStage;
            next = next + kStage == kRing ? 0 : next + kStage;
        }
        wait<0>();
        if constexpr (WK > 1) {
            // each wave's sums into its own ring (no load is in flight there any more)
            constexpr int kTiles = TN / 16 * (TM / 16);
            static_assert(kTiles * 1024 <= kRing, "the sums fit the ring");
            Acc *mine = reinterpret_cast<Acc *>(lds) + lane_id();
#pragma unroll
            for (int n = 0; n < TN / 16; ++n)
#pragma unroll
                for (int m = 0; m < TM / 16; ++m) mine[(n * (TM / 16) + m) * 64] = acc[n][m];
            __syncthreads();
            if (first == 0) {
#pragma unroll
                for (int n = 0; n < TN / 16; ++n)
#pragma unroll
                    for (int m = 0; m < TM / 16; ++m)
#pragma unroll
                        for (int q = 1; q < WK; ++q)
                            acc[n][m] += mine[q * (kRing / 16) + (n * (TM / 16) + m) * 64];
            }
        }
    }

    // Stores the tile: scaled(row, col, v) may change the four values from column col of row
    // on (within the tile), and what lies in the first `rows` rows and `cols` columns goes to
    // out, `ld` elements from row to row.
    //
    // The sums lie four to a lane, so straight from them a store would touch 32 or 64 bytes
    // of each of 16 rows. The wave's tile passes through its own part of the ring instead, as
    // many rows at a time as fit, and a store takes whole rows of it: 128 bytes (bf16) or 256
    // of each row with TN = 64, whole lines. Rows are 16 bytes longer in the ring, so that 16
    // lanes which write one column of 16 rows hit different banks.
    //
    // stream: past the caches, for outputs that they cannot hold until they are read (a
    // million rows 1024 -> 4096, 8.6 GB: 8.2 ms instead of 8.7; 44625 rows 24 -> 744, 66 MB, the
    // other way: 39 us instead of 26).
    template <bool OUT_BF16, typename F>
    __device__ static void put(char *lds, Sums &acc, int rows, int cols, void *out, int64_t ld,
                               bool stream, F &&scaled) {
        constexpr int OB = OUT_BF16 ? 2 : 4, E = 16 / OB;  // bytes of an element, elements of a store
        constexpr int kLine = TN * OB + 16, kOwn = kRing / (WM * WN);
        constexpr int kFit = kOwn / (16 * kLine), kAll = TM / 16;
        constexpr int MT = kFit >= kAll ? kAll : kFit >= 4 ? 4 : kFit >= 2 ? 2 : 1;
        static_assert(kFit >= 1 && kAll % MT == 0, "the wave's part of the ring");
        constexpr int kAcross = TN / E, kDown = 64 / kAcross;
        char *own = lds + (WK > 1 ? 0 : wave_id()) * kOwn;
        const int l = lane_id(), down = l / kAcross, across = l % kAcross * E;
#pragma unroll
        for (int m0 = 0; m0 < kAll; m0 += MT) {
            if (m0 > 0) wave_order();  // the rows before have been read
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < TN / 16; ++n) {
                    const int row = m * 16 + (l & 15), col = n * 16 + (l >> 4) * 4;
                    float v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = (float)acc[n][m0 + m][j];
                    scaled(row0() + m0 * 16 + row, col0() + col, v);
                    char *to = own + row * kLine + col * OB;
                    if constexpr (OUT_BF16)
                        *reinterpret_cast<v2u *>(to) =
                            v2u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                    else
                        *reinterpret_cast<v4f *>(to) = v4f{v[0], v[1], v[2], v[3]};
                }
            wave_order();
#pragma unroll
            for (int i = 0; i < MT * 16 / kDown; ++i) {
                const int at = i * kDown + down, row = row0() + m0 * 16 + at, col = col0() + across;
                const v4u q = *reinterpret_cast<const v4u *>(own + at * kLine + across * OB);
                v4u *to = reinterpret_cast<v4u *>(static_cast<char *>(out) + (row * ld + col) * OB);
                if (row < rows && col < cols) store_streamed(q, to, stream);
            }
        }
    }
};

}  // namespace tiles
}  // namespace moonep
