// Rows in microscaled 4-bit floating point and the experts' products of them, for gfx950.
//
// 32 values next to each other are e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and their
// negatives, two to a byte, the even one low) with one scale, a byte that stands for
// 2^(byte - 127) and for NaN at 255.
//
//   y[t][n] = sum over blocks b of 2^(sx[t][b] + sw[n][b] - 254) sum_{i in b} x[t,i] w[n,i]
//
// which is what the matrix units' scaled instruction adds up: a lane's 16 bytes are one
// block, and it brings the block's scale along.
#include "emit.h"
#include "layerops.h"
#include "segments.h"
#include "tiles.h"

namespace moonep {
namespace {

using namespace emit;
using namespace segments;

constexpr int kThreads = 256;

// LANES lanes to a row, U chunks of 16 bytes a lane on their way at a time.
template <bool BF16, int LANES, int U>
__global__ __launch_bounds__(kThreads) void k_quantize_mx(int64_t first, int64_t n_rows, int chunks,
                                                          const v4u *x, uint8_t *q, uint8_t *scale,
                                                          bool stream) {
    constexpr int N = Chunk<BF16>::N, kRows = kThreads / LANES;
    const int lane = threadIdx.x % LANES;
    const int64_t row = first + (int64_t)blockIdx.x * kRows + threadIdx.x / LANES;
    if (row >= n_rows) return;
    const int64_t cols = (int64_t)chunks * N;
    x += row * chunks;
    q += row * (cols / 2);
    scale += row * scale_pitch(cols);
    // whole groups of lanes, so that the blocks' lanes are all there
    for (int c0 = 0; c0 < chunks; c0 += LANES * U) {
        v4u v[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int c = c0 + i * LANES + lane;
            v[i] = v4u{0, 0, 0, 0};
            if (c < chunks) v[i] = __builtin_nontemporal_load(x + c);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float f[N];
            Chunk<BF16>::unpack(v[i], f);
            put4<N>(f, c0 + i * LANES + lane, chunks, stream, q, scale);
        }
    }
}

template <bool BF16, int LANES, int U>
hipError_t quantize_rows(int64_t n_rows, int chunks, const void *x, uint8_t *q, uint8_t *scale,
                         hipStream_t st) {
    constexpr int64_t kPiece = launch_groups(kThreads), kRows = kThreads / LANES;
    const bool stream = n_rows * chunks * Chunk<BF16>::N / 2 >= kStreamBytes;
    for (int64_t at = 0; at < n_rows; at += kPiece * kRows) {
        const int64_t wgs = (n_rows - at + kRows - 1) / kRows;
        hipLaunchKernelGGL((k_quantize_mx<BF16, LANES, U>), dim3((unsigned)(wgs < kPiece ? wgs : kPiece)),
                           dim3(kThreads), 0, st, at, n_rows, chunks, static_cast<const v4u *>(x), q,
                           scale, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// A wave for rows of up to 256 chunks, a workgroup for longer ones. Gigabytes of bf16, us:
//   262144 x 2048 (256 chunks)   64 lanes 232, 256 lanes 268
//   130944 x 4096                         210           207
//   131072 x 7168                         411           360 (2.4 GB, 6.7 TB/s)
// Short rows: 1048576 of 64 columns 8 lanes 35, 16 lanes of two chunks 58.
template <bool BF16>
hipError_t quantize(int64_t n_rows, int chunks, const void *x, uint8_t *q, uint8_t *scale,
                    hipStream_t st) {
    if (chunks <= 8) return quantize_rows<BF16, 8, 1>(n_rows, chunks, x, q, scale, st);
    if (chunks <= 32) return quantize_rows<BF16, 16, 2>(n_rows, chunks, x, q, scale, st);
    if (chunks <= 256) return quantize_rows<BF16, 64, 2>(n_rows, chunks, x, q, scale, st);
    return quantize_rows<BF16, 256, 1>(n_rows, chunks, x, q, scale, st);
}

// ------------------------------------------------------------------ products

typedef int v8i __attribute__((ext_vector_type(8)));

// 64 lanes x 4 bytes from the buffer at voff into shared memory at `to` onwards.
__device__ __forceinline__ void load_words_to_lds(uint32_t to, int voff, __amdgpu_buffer_rsrc_t rs) {
    asm volatile("s_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"{m0}"(to), "v"(voff), "s"(rs)
                 : "memory");
}

// A tile of the product (tiles.h) whose steps are 128 bytes of a row, 256 values, and its rows'
// scales, 8 bytes a step, in rings of their own behind the parts'.
//
// 262144 rows of 64 segments, 2048 -> 1024, take 386 to 400 us, 2.8 PFLOP/s of the 7.9 that the
// instruction reaches from registers, and from 7168 columns 1162, 3.3: a tile of 256 x 256 takes
// 2.3 us a step and 5 besides (its segment's look-up, the first loads, the store). The matrix units
// are busy a third of the time; shared memory has 192 KB of fragments read for 64 KB loaded a
// step. Fragments read a group ahead of their products (446 us, when this took 409), steps of
// half the length (484), workgroups that go on to further tiles (412 to 413), the next tile's rows
// brought to L2, another order along k and wave priorities were no faster.
//
// WIDE: rows are whole groups of 512 values, so a lane loads a row's scales of two steps, 16
// bytes, at once: each load of a step's scales alone touches a line of every row, as many lines
// as the parts themselves. It reads them from shared memory at once too, and the instruction
// takes a byte of a register for each half of the two steps (410 us with a read of a byte for
// each). Else a lane loads the 4 bytes of half a step, word h * BT + row, and
// bytes behind a row's last block, which may hold anything, are masked (256 segments of 250 rows to
// 1024 columns: 179 us from 2080 columns, WIDE 128 from 2048).
template <int BM, int BN, int WM, int WN, int STAGES, bool WIDE>
struct ScaledProduct : tiles::Product<2, false, false, BM, BN, WM, WN, 1, STAGES> {
    typedef tiles::Product<2, false, false, BM, BN, WM, WN, 1, STAGES> Base;
    typedef typename Base::X X;
    typedef typename Base::W W;
    typedef typename Base::Sums Sums;
    static constexpr int NW = WM * WN, TM = Base::TM, TN = Base::TN;
    static constexpr int kSteps = WIDE ? 2 : 1;            // that a load of scales serves
    static constexpr int kLane = WIDE ? 16 : 4;            // bytes of a lane's load
    static constexpr int kPart = (BM + BN) * 8 * kSteps;   // bytes of all rows' scales for them
    static constexpr int kScaleLoads = (kPart / kLane + NW * 64 - 1) / (NW * 64);  // of a wave
    static constexpr int kOwn = kScaleLoads * NW * 64 * kLane;  // kPart and what idle lanes load
    static constexpr int kParts = WIDE ? STAGES / 2 + 1 : STAGES;
    static constexpr int kLds = STAGES * Base::kStage + kParts * kOwn;
    static_assert(BM % 64 == 0, "a wave's load is of one operand's rows");

    struct Scales {
        const char *x, *w;     // first row of the tile's
        int x_bytes, w_bytes;  // up to the operands' ends
        int pitch;
        int voff[kScaleLoads], in_step[kScaleLoads];
        bool of_x[kScaleLoads];

        __device__ void init(const void *px, int x_rows, const void *pw, int w_rows, int pitch_) {
            x = static_cast<const char *>(px);
            w = static_cast<const char *>(pw);
            pitch = pitch_;
            x_bytes = x_rows * pitch;
            w_bytes = w_rows * pitch;
            constexpr int kXLanes = WIDE ? BM : 2 * BM, kAll = WIDE ? BM + BN : 2 * (BM + BN);
#pragma unroll
            for (int i = 0; i < kScaleLoads; ++i) {
                const int at = (i * NW + tiles::wave_id()) * 64 + lane_id();
                of_x[i] = at < kXLanes;
                const int in = of_x[i] ? at : at - kXLanes, bt = of_x[i] ? BM : BN;
                in_step[i] = at < kAll ? in / bt * 4 : tiles::kOutOfRange;
                voff[i] = in % bt * pitch + (at < kAll ? in_step[i] : 0);
            }
        }

        // The scales from step s on (WIDE: an even one) to `to`.
        __device__ void load(int s, uint32_t to) {
            const int at = s * 8, left = pitch - at;  // bytes of a row from the step on
#pragma unroll
            for (int i = 0; i < kScaleLoads; ++i) {
                const uint32_t mine = to + (i * NW + tiles::wave_id()) * 64 * kLane;
                const int off = in_step[i] < left ? voff[i] : tiles::kOutOfRange;
                const bool first = __builtin_amdgcn_readfirstlane(of_x[i]);
                const __amdgpu_buffer_rsrc_t rs =
                    tiles::rsrc((first ? x : w) + at, max((first ? x_bytes : w_bytes) - at, 0));
                if constexpr (WIDE) tiles::load_to_lds<0>(mine, off, rs);
                else load_words_to_lds(mine, off, rs);
            }
        }
    };

    // Byte H of the words sw and sx is the scale of this lane's block.
    template <int H>
    __device__ static v4f mma(const v4u &w, const v4u &x, v4f c, uint32_t sw, uint32_t sx) {
        const v8i a = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
        const v8i b = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, H, (int)sw, H, (int)sx);
    }

    // cols: values of a row of k. The rest as Product::run.
    __device__ static void run(X &x, W &w, Scales &sc, int cols, int rows, char *lds, Sums &acc) {
        const bool busy = Base::row0() < rows;
        const int steps = (cols + 255) / 256, blocks = cols / 32;
        const uint32_t base = tiles::lds_offset(lds);
        const int l = lane_id(), g = l >> 4;
        constexpr int kScalesAt = STAGES * Base::kStage;
#pragma unroll
        for (int n = 0; n < TN / 16; ++n)
#pragma unroll
            for (int m = 0; m < TM / 16; ++m) acc[n][m] = v4f{0, 0, 0, 0};
        // The scales go first, so that they are there when their step's parts are.
        auto load = [&](int s, uint32_t to) {
            if (!WIDE || s % 2 == 0) sc.load(s, base + kScalesAt + s / kSteps % kParts * kOwn);
            x.load(s, to);
            w.load(s, to + X::kBytes);
        };
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) load(s, base + s * Base::kStage);
        int at = 0, next = (STAGES - 1) * Base::kStage;
        uint32_t sx[TM / 16], sw[TN / 16];  // WIDE: a byte for each half of two steps
        for (int s0 = 0; s0 < steps; s0 += kSteps)
            tiles::each<kSteps>([&](auto sub) {
                constexpr int S = decltype(sub)::value;
                const int s = s0 + S;
                // scales in flight beside the parts only make this wait longer
                Base::template wait<(STAGES - 2) * Base::kLoads>();
                // steps past the last one load nothing: their range is empty
                load(s + STAGES - 1, base + next);
                const char *part = lds + at;
                const char *scales = lds + kScalesAt + s / kSteps % kParts * kOwn;
                at = at + Base::kStage == STAGES * Base::kStage ? 0 : at + Base::kStage;
                next = next + Base::kStage == STAGES * Base::kStage ? 0 : next + Base::kStage;
                if (!busy) return;
                if constexpr (WIDE && S == 0) {
                    auto all = [&](int row) {
                        const v4u t = *reinterpret_cast<const v4u *>(scales + (row + (l & 15)) * 16);
                        const uint32_t mine = g | (4 + g) << 8;
                        return __builtin_amdgcn_perm(__builtin_amdgcn_perm(t.w, t.z, mine),
                                                     __builtin_amdgcn_perm(t.y, t.x, mine), 0x05040100u);
                    };
#pragma unroll
                    for (int n = 0; n < TN / 16; ++n) sw[n] = all(BM + Base::col0() + n * 16);
#pragma unroll
                    for (int m = 0; m < TM / 16; ++m) sx[m] = all(Base::row0() + m * 16);
                }
                tiles::each<2>([&](auto half) {
                    constexpr int h = decltype(half)::value;
                    v4u fx[TM / 16], fw[TN / 16];
                    const int mask = s * 8 + h * 4 + g < blocks ? 0xff : 0;
                    auto byte = [&](int word) { return *(const uint8_t *)(scales + (word + (l & 15)) * 4 + g) & mask; };
#pragma unroll
                    for (int n = 0; n < TN / 16; ++n) {
                        fw[n] = __builtin_bit_cast(v4u, W::read(part + X::kBytes, Base::col0() + n * 16, h));
                        if constexpr (!WIDE) sw[n] = byte(2 * BM + h * BN + Base::col0() + n * 16);
                    }
#pragma unroll
                    for (int m = 0; m < TM / 16; ++m) {
                        fx[m] = __builtin_bit_cast(v4u, X::read(part, Base::row0() + m * 16, h));
                        if constexpr (!WIDE) sx[m] = byte(h * BM + Base::row0() + m * 16);
                    }
#pragma unroll
                    for (int n = 0; n < TN / 16; ++n)
#pragma unroll
                        for (int m = 0; m < TM / 16; ++m)
                            acc[n][m] = mma<WIDE ? S * 2 + h : 0>(fw[n], fx[m], acc[n][m], sw[n], sx[m]);
                });
            });
        Base::template wait<0>();
    }
};

struct ScaledArgs {
    const uint8_t *x, *x_scale, *w, *w_scale, *dup_w, *dup_scale;
    void *y;
};

template <typename P, bool OUT_BF16, int BM, int BN>
__global__ __launch_bounds__(P::kThreads) void k_matmul_mx(ExpertShape sh, const int32_t *seg_ptr,
                                                            ScaledArgs a, Order order, uint32_t first,
                                                            bool stream) {
    __shared__ __align__(1024) char lds[P::kLds];
    const Place at = place(order, first);
    if (at.unit < 0) return;
    const int r = at.unit;
    const Tile t = find_tile(seg_ptr + (int64_t)r * (sh.n_seg + 1), sh.G + sh.B, sh.SK, BM, at.m);
    if (t.seg < 0) return;
    const bool home = t.seg < sh.G;
    const int64_t which = home ? (int64_t)r * sh.G + t.seg : (int64_t)r * sh.slots + t.seg - sh.G;
    const int64_t row0 = (int64_t)r * sh.SK + t.row;
    const int n0 = at.n * BN, n_rows = min(BN, sh.n_out - n0);
    const int row = sh.n_in / 2, pitch = scale_pitch(sh.n_in);
    typename P::X px;
    typename P::W pw;
    typename P::Scales sc;
    px.init((const char *)a.x + row0 * row, row, t.rows, 0);
    pw.init((const char *)(home ? a.w : a.dup_w) + which * sh.block + (int64_t)n0 * row, row, n_rows, 0);
    sc.init(a.x_scale + row0 * pitch, t.rows,
            (home ? a.w_scale : a.dup_scale) + which * sh.scale_block + (int64_t)n0 * pitch, n_rows,
            pitch);
    typename P::Sums acc;
    P::run(px, pw, sc, sh.n_in, t.rows, lds, acc);
    char *out = static_cast<char *>(a.y) + (row0 * sh.n_out + n0) * (OUT_BF16 ? 2 : 4);
    P::template put<OUT_BF16>(lds, acc, t.rows, sh.n_out - n0, out, sh.n_out, stream,
                              [](int, int, float *) {});
}

template <bool OUT_BF16, int BM, int BN, int WM, int WN, int STAGES, bool WIDE>
hipError_t matmul_tiles_of(const ExpertShape &sh, const int32_t *seg_ptr, const ScaledArgs &a,
                           hipStream_t st) {
    typedef ScaledProduct<BM, BN, WM, WN, STAGES, WIDE> P;
    const int64_t tm = most_tiles(sh, BM), tn = tiles_of(sh.n_out, BN);
    const bool stream = (int64_t)sh.R * sh.SK * sh.n_out * (OUT_BF16 ? 2 : 4) >= kStreamBytes;
    return in_order(sh.R, tm, tn, 8, sh.R % 8 == 0, [&](const Order &order, uint32_t at, dim3 grid) {
        hipLaunchKernelGGL((k_matmul_mx<P, OUT_BF16, BM, BN>), grid, dim3(P::kThreads), 0, st, sh,
                           seg_ptr, a, order, at, stream);
    });
}

template <bool OUT_BF16, int BM, int BN, int WM, int WN, int STAGES>
hipError_t matmul_tiles(const ExpertShape &sh, const int32_t *seg_ptr, const ScaledArgs &a,
                        hipStream_t st) {
    // scales of a matrix lie on 16 bytes where their distance says so
    if (sh.n_in % 512 == 0 && sh.scale_block % 16 == 0)
        return matmul_tiles_of<OUT_BF16, BM, BN, WM, WN, STAGES, true>(sh, seg_ptr, a, st);
    return matmul_tiles_of<OUT_BF16, BM, BN, WM, WN, STAGES, false>(sh, seg_ptr, a, st);
}

// The tile by the rows that a segment has on average (half the duplicate slots counted as used)
// and the tiles that makes. 256 segments, 2048 -> 1024 columns, us:
//   rows      64x64 (3 stages)  64x128 (3)  128x128 (2)  128x256 (3)  256x256 (2)
//      16           71              57           65           59          70
//      64          102              78           78           77          81
//     100          133              96           90           84          87
//     150          189             133          123          110         100
//     250          273             195          157          146         130
//     500          506             358          287          273         228
// 16 of 10 rows, 4096 -> 1024: 64x64 11.6, 64x128 14.6, 128x256 16.8. The change to 256x256 is set
// for segments that are much alike: 256 of 128 rows, 7168 -> 512, 155 with it and 163 with 128x256.
// Skewed ones, which the host cannot see, lose by it there: 1152 of 2 to 622 rows, 128 by this
// estimate, 7168 -> 512, 675 and 650.
template <bool OUT_BF16>
hipError_t matmul(const ExpertShape &sh, const int32_t *seg_ptr, const ScaledArgs &a, hipStream_t st) {
    const int64_t segs = sh.G + sh.B / 2 < sh.SK ? sh.G + sh.B / 2 : sh.SK;
    const int64_t rows = tiles_of(sh.SK, (int)segs);
    auto tiles = [&](int bm, int bn) { return sh.R * segs * tiles_of(rows, bm) * tiles_of(sh.n_out, bn); };
    if (sh.n_out > 128 && rows >= 128 && fills(tiles(256, 256)))
        return matmul_tiles<OUT_BF16, 256, 256, 2, 4, 2>(sh, seg_ptr, a, st);
    if (sh.n_out > 128 && rows >= 32 && fills(tiles(128, 256)))
        return matmul_tiles<OUT_BF16, 128, 256, 2, 4, 3>(sh, seg_ptr, a, st);
    if (sh.n_out > 64 && tiles(64, 128) >= kFill)
        return matmul_tiles<OUT_BF16, 64, 128, 2, 2, 3>(sh, seg_ptr, a, st);
    return matmul_tiles<OUT_BF16, 64, 64, 2, 2, 3>(sh, seg_ptr, a, st);
}

}  // namespace

hipError_t launch_quantize_rows_mx(int64_t n_rows, int32_t cols, const void *x, int bf16,
                                    uint8_t *q, uint8_t *scale, hipStream_t st) {
    return bf16 ? quantize<true>(n_rows, cols / 8, x, q, scale, st)
                : quantize<false>(n_rows, cols / 4, x, q, scale, st);
}

hipError_t launch_expert_matmul_mx(const ExpertShape &sh, const int32_t *seg_ptr, const uint8_t *x,
                                    const uint8_t *x_scale, const uint8_t *w, const uint8_t *w_scale,
                                    const uint8_t *dup_w, const uint8_t *dup_scale, void *y,
                                    int y_bf16, hipStream_t st) {
    const ScaledArgs a = {x, x_scale, w, w_scale, dup_w, dup_scale, y};
    return y_bf16 ? matmul<true>(sh, seg_ptr, a, st) : matmul<false>(sh, seg_ptr, a, st);
}

}  // namespace moonep
