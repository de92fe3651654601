// One output tile of a matrix product on the matrix units of gfx950, for the
// experts' products (experts.hip). Not part of the ABI.
//
// D[m][n] = sum_k X[m][k] W[n][k]. A workgroup holds the tile's sums in registers
// and walks k in steps of 128 bytes of a row: both operands' parts of a step are
// loaded straight into shared memory (16 bytes a lane, no registers on the way),
// kStages - 1 steps ahead of the one the matrix units work on, with one barrier for
// each step.
//
// An operand lies in memory in one of two ways:
//   rows   k runs along its rows: the step's part is [BT][128 bytes]
//   cols   k runs across its rows: the step's part is [128 / EB rows of k][BT elements],
//          and lanes get their k values with transposing reads (2-byte elements) or one
//          by one (4-byte elements)
// The 16-byte chunks of a part's rows are exchanged by an XOR with some of the row's
// bits, so that lanes which read the same chunk of different rows hit different banks.
// Loads past the operand's end (rows behind a segment, the last step's k, columns behind
// the matrix) return zeros by the buffer's range check, or land in sums that are not
// stored.
#pragma once

#include <type_traits>

#include "rows.h"

namespace moonep {
namespace tiles {

using namespace rows;

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kStepBytes = 128;
constexpr int kOutOfRange = 0x7ffffff0;

__device__ __forceinline__ uint32_t lds_offset(const void *p) {
    return (uint32_t)(uintptr_t)(const lds_char *)p;
}

// 64 lanes x 16 bytes from the buffer at voff into shared memory at `to` onwards, lane
// after lane. Done when vmcnt says so.
__device__ __forceinline__ void load_to_lds(uint32_t to, int voff, __amdgpu_buffer_rsrc_t rs) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to),
        "v"(voff), "s"(rs)
        : "memory", "m0");
}

__device__ __forceinline__ int wave_id() {
    return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
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
template <int EB, bool COLS, int BT, int NW>
struct Side {
    static constexpr int kBytes = BT * kStepBytes;  // of one step's part
    static constexpr int kLoads = BT / 8 / NW;      // by each wave
    static constexpr int kK = kStepBytes / EB;      // k of one step
    static constexpr int kRow = COLS ? BT * EB : kStepBytes;
    static constexpr int kChunks = kRow / 16;
    static_assert(BT % (8 * NW) == 0, "each wave loads whole kilobytes");

    __device__ static int wave() { return NW == 1 ? 0 : wave_id(); }

    __device__ static int swizzle(int row) {
        if constexpr (!COLS) return (row >> 1) & 7;
        if constexpr (EB == 4) return ((row >> 2) & 3) << 2;
        if constexpr (kChunks >= 16) return ((row & 3) | ((row >> 3) & 1) << 2) << 1;
        if constexpr (kChunks == 8) return (((row >> 1) & 1) | ((row >> 3) & 1) << 1) << 1;
        return ((row >> 3) & 1) << 1;
    }

    const char *base;  // first element of the tile
    int ld, left;      // bytes of a row; rows: bytes from base to the operand's end,
                       // cols: bytes of a row before base
    int k;             // cols: rows of k
    int voff[kLoads], chunk[COLS ? 1 : kLoads];

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
            if constexpr (!COLS) chunk[i] = c * 16;
        }
    }

    __device__ void load(int step, uint32_t to) {
        const uint32_t mine = to + wave() * 1024;
        if constexpr (COLS) {
            const int rows = min(k - step * kK, kK);
            const auto rs = rsrc(base + (int64_t)step * kK * ld, rows > 0 ? rows * ld - left : 0);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) load_to_lds(mine + i * NW * 1024, voff[i], rs);
        } else {
            const int at = step * kStepBytes;
            const auto rs = rsrc(base + at, max(left - at, 0));
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                load_to_lds(mine + i * NW * 1024, chunk[i] < ld - at ? voff[i] : kOutOfRange, rs);
        }
    }

    // Fragments of 16 rows from row `first` on, half `h` of the step.
    typedef typename Unit<EB>::Frag Frag;
    template <int N>
    __device__ static void read(const char *part, int first, int h, Frag *f) {
        const int l = lane_id(), i = l & 15, g = l >> 4;
        if constexpr (!COLS) {
            const char *p = part + (first + i) * kRow + (((h * 4 + g) ^ swizzle(i)) * 16);
#pragma unroll
            for (int t = 0; t < N; ++t) f[t] = *reinterpret_cast<const Frag *>(p + t * 16 * kRow);
        } else if constexpr (EB == 2) {
            const int row = g * 8 + (i >> 2);
#pragma unroll
            for (int t = 0; t < N; ++t) {
                const int c = first / 8 + t * 2 + ((i >> 1) & 1);
                const char *p = part + h * 32 * kRow + row * kRow + (c ^ swizzle(row)) * 16 + (i & 1) * 8;
                typedef __attribute__((address_space(3))) v4s lds_v4s;
                const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)p);
                const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(p + 4 * kRow));
                f[t] = __builtin_bit_cast(Frag, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            }
        } else {
            const int row = g * 4;
#pragma unroll
            for (int t = 0; t < N; ++t) {
                const int c = first / 4 + t * 4 + (i >> 2);
                const char *p = part + h * 16 * kRow + row * kRow + (c ^ swizzle(row)) * 16 + (i & 3) * 4;
#pragma unroll
                for (int j = 0; j < 4; ++j) f[t][j] = *reinterpret_cast<const float *>(p + j * kRow);
            }
        }
    }
};

// The tile's sums. Wave w of WM x WN holds rows (w % WM) * TM .. and columns
// (w / WM) * TN ..; lane l of acc[n][m] holds row m * 16 + l % 16 and the four columns from
// n * 16 + l / 16 * 4 on: the columns go into the matrix unit's first operand, so that a
// lane's four sums lie side by side in an output row.
//
// With WK > 1 every wave makes the whole tile over every WK-th step, in shared memory of
// its own and without barriers; the waves' sums are added in the waves' order at the end,
// and wave 0 holds the tile.
template <int EB, bool XCOLS, bool WCOLS, int BM, int BN, int WM, int WN, int WK, int STAGES>
struct Product {
    static_assert(WK == 1 || WM * WN == 1, "waves share a tile or the steps");
    static constexpr int kThreads = WM * WN * WK * 64;
    static constexpr int TM = BM / WM, TN = BN / WN;
    typedef Side<EB, XCOLS, BM, WM * WN> X;
    typedef Side<EB, WCOLS, BN, WM * WN> W;
    static constexpr int kStage = X::kBytes + W::kBytes;
    static constexpr int kRing = STAGES * kStage;  // shared memory of the waves of one tile
    static constexpr int kLds = WK * kRing;
    static constexpr int kLoads = X::kLoads + W::kLoads;
    typedef typename Unit<EB>::Acc Acc;
    typedef Acc Sums[TN / 16][TM / 16];

    __device__ static int row0() { return WK > 1 ? 0 : wave_id() % WM * TM; }
    __device__ static int col0() { return WK > 1 ? 0 : wave_id() / WM * TN; }
    __device__ static bool holds() { return WK == 1 || wave_id() == 0; }

    // At most N loads in flight, and what the tile's waves loaded is there for all of them.
    template <int N>
    __device__ static void wait() {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
        if constexpr (WK == 1) __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }

    __device__ static void run(X &x, W &w, int k, char *lds, Sums &acc) {
        const int first = WK > 1 ? wave_id() : 0;
        const int steps = (k + X::kK - 1) / X::kK;
        lds += first * kRing;
        const uint32_t base = lds_offset(lds);
#pragma unroll
        for (int n = 0; n < TN / 16; ++n)
#pragma unroll
            for (int m = 0; m < TM / 16; ++m) acc[n][m] = Acc{0, 0, 0, 0};
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
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                typename X::Frag fx[TM / 16], fw[TN / 16];
                W::template read<TN / 16>(part + X::kBytes, col0(), h, fw);
                X::template read<TM / 16>(part, row0(), h, fx);
#pragma unroll
                for (int n = 0; n < TN / 16; ++n)
#pragma unroll
                    for (int m = 0; m < TM / 16; ++m)
                        acc[n][m] = Unit<EB>::mma(fw[n], fx[m], acc[n][m]);
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
};

}  // namespace tiles
}  // namespace moonep
