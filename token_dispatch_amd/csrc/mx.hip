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

// One chunk of 16 bytes a lane at a time, LANES lanes to a row.
template <bool BF16, int LANES>
__global__ __launch_bounds__(kThreads) void k_quantize_mx(int64_t first, int64_t n_rows, int chunks,
                                                           const v4u *x, uint8_t *q, uint8_t *scale,
                                                           bool stream) {
    constexpr int N = Chunk<BF16>::N, kRows = kThreads / LANES;
    const int lane = threadIdx.x % LANES;
    const int64_t row = first + (int64_t)blockIdx.x * kRows + threadIdx.x / LANES;
    if (row >= n_rows) return;
    const int64_t cols = (int64_t)chunks * N;
    q += row * (cols / 2);
    scale += row * scale_pitch(cols);
    // whole groups of lanes, so that the blocks' lanes are all there
    for (int c = lane; c - lane < chunks; c += LANES) {
        float v[N] = {};
        if (c < chunks) Chunk<BF16>::unpack(__builtin_nontemporal_load(x + row * chunks + c), v);
        put4<N>(v, c, chunks, stream, q, scale);
    }
}

template <bool BF16, int LANES>
hipError_t quantize_rows(int64_t n_rows, int chunks, const void *x, uint8_t *q, uint8_t *scale,
                         hipStream_t st) {
    constexpr int64_t kPiece = (int64_t)1 << 22, kRows = kThreads / LANES;
    const bool stream = n_rows * chunks * Chunk<BF16>::N / 2 >= kStreamBytes;
    for (int64_t at = 0; at < n_rows; at += kPiece * kRows) {
        const int64_t wgs = (n_rows - at + kRows - 1) / kRows;
        hipLaunchKernelGGL((k_quantize_mx<BF16, LANES>), dim3((unsigned)(wgs < kPiece ? wgs : kPiece)),
                           dim3(kThreads), 0, st, at, n_rows, chunks, static_cast<const v4u *>(x), q,
                           scale, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <bool BF16>
hipError_t quantize(int64_t n_rows, int chunks, const void *x, uint8_t *q, uint8_t *scale,
                    hipStream_t st) {
    if (chunks <= 32) return quantize_rows<BF16, 16>(n_rows, chunks, x, q, scale, st);
    if (chunks <= 128) return quantize_rows<BF16, 64>(n_rows, chunks, x, q, scale, st);
    return quantize_rows<BF16, 256>(n_rows, chunks, x, q, scale, st);
}

// ------------------------------------------------------------------ products

typedef int v8i __attribute__((ext_vector_type(8)));

// 64 lanes x 4 bytes from the buffer at voff into shared memory at `to` onwards.
__device__ __forceinline__ void load_words_to_lds(uint32_t to, int voff, __amdgpu_buffer_rsrc_t rs) {
    asm volatile("s_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"{m0}"(to), "v"(voff), "s"(rs)
                 : "memory");
}

// A tile of the product (tiles.h) whose steps are 128 bytes of a row, 256 values. Beside an
// operand's part of a step its rows' 8 scales lie in the ring, four of them (half a step's)
// to a word: word h * BT + row. A wave loads kScaleLoads times 64 words; loads past the last
// ones land behind them.
template <int BM, int BN, int WM, int WN, int STAGES>
struct ScaledProduct : tiles::Product<2, false, false, BM, BN, WM, WN, 1, STAGES> {
    typedef tiles::Product<2, false, false, BM, BN, WM, WN, 1, STAGES> Base;
    typedef typename Base::X X;
    typedef typename Base::W W;
    typedef typename Base::Sums Sums;
    static constexpr int NW = WM * WN;
    static constexpr int kWords = 2 * (BM + BN), kXWords = 2 * BM;
    static constexpr int kScaleLoads = (kWords / 64 + NW - 1) / NW;
    static constexpr int kScaleStage = kScaleLoads * NW * 256;
    static constexpr int kStage = Base::kStage + kScaleStage;
    static constexpr int kLds = STAGES * kStage;
    static constexpr int kLoads = Base::kLoads + kScaleLoads;
    static constexpr int TM = Base::TM, TN = Base::TN;
    static_assert(kXWords % 64 == 0 && kWords % 64 == 0, "a load's words are one operand's");

    struct Scales {
        const char *x, *w;     // first row of the tile's
        int x_bytes, w_bytes;  // up to the operands' ends
        int pitch;
        int voff[kScaleLoads], half[kScaleLoads];

        __device__ void init(const void *px, int x_rows, const void *pw, int w_rows, int pitch_) {
            x = static_cast<const char *>(px);
            w = static_cast<const char *>(pw);
            pitch = pitch_;
            x_bytes = x_rows * pitch;
            w_bytes = w_rows * pitch;
#pragma unroll
            for (int i = 0; i < kScaleLoads; ++i) {
                const int at = (i * NW + tiles::wave_id()) * 64 + lane_id();
                const bool of_x = at < kXWords;
                const int in = of_x ? at : at - kXWords, bt = of_x ? BM : BN;
                half[i] = in < 2 * bt ? in / bt * 4 : tiles::kOutOfRange;
                voff[i] = in % bt * pitch + (in < 2 * bt ? half[i] : 0);
            }
        }

        __device__ void load(int s, uint32_t to) {
            const int at = s * 8, left = pitch - at;  // bytes of a row from the step on
#pragma unroll
            for (int i = 0; i < kScaleLoads; ++i) {
                const int q = i * NW + tiles::wave_id();
                const bool of_x = q * 64 < kXWords;
                const __amdgpu_buffer_rsrc_t rs =
                    tiles::rsrc((of_x ? x : w) + at, max((of_x ? x_bytes : w_bytes) - at, 0));
                load_words_to_lds(to + q * 256, half[i] < left ? voff[i] : tiles::kOutOfRange, rs);
            }
        }
    };

    __device__ static v4f mma(const v4u &w, const v4u &x, v4f c, int sw, int sx) {
        const v8i a = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
        const v8i b = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, 0, sw, 0, sx);
    }

    // cols: values of a row of k. The rest as Product::run.
    __device__ static void run(X &x, W &w, Scales &sc, int cols, int rows, char *lds, Sums &acc) {
        const bool busy = Base::row0() < rows;
        const int steps = (cols + 255) / 256, blocks = cols / 32;
        const uint32_t base = tiles::lds_offset(lds);
        const int l = lane_id(), g = l >> 4;
#pragma unroll
        for (int n = 0; n < TN / 16; ++n)
#pragma unroll
            for (int m = 0; m < TM / 16; ++m) acc[n][m] = v4f{0, 0, 0, 0};
        auto load = [&](int s, uint32_t to) {
            x.load(s, to);
            w.load(s, to + X::kBytes);
            sc.load(s, to + Base::kStage);
        };
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) load(s, base + s * kStage);
        int at = 0, next = (STAGES - 1) * kStage;
        for (int s = 0; s < steps; ++s) {
            Base::template wait<(STAGES - 2) * kLoads>();
            // steps past the last one load nothing: their range is empty
            load(s + STAGES - 1, base + next);
            const char *part = lds + at;
            if (busy) {
                const char *scales = part + Base::kStage + (l & 15) * 4 + g;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // bytes behind a row's last block may hold anything, NaN among it
                    const int mask = s * 8 + h * 4 + g < blocks ? 0xff : 0;
                    v4u fx[TM / 16], fw[TN / 16];
                    int sx[TM / 16], sw[TN / 16];
#pragma unroll
                    for (int n = 0; n < TN / 16; ++n) {
                        fw[n] = __builtin_bit_cast(v4u, W::read(part + X::kBytes, Base::col0() + n * 16, h));
                        sw[n] = *(const uint8_t *)(scales + (kXWords + h * BN + Base::col0() + n * 16) * 4) & mask;
                    }
#pragma unroll
                    for (int m = 0; m < TM / 16; ++m) {
                        fx[m] = __builtin_bit_cast(v4u, X::read(part, Base::row0() + m * 16, h));
                        sx[m] = *(const uint8_t *)(scales + (h * BM + Base::row0() + m * 16) * 4) & mask;
                    }
#pragma unroll
                    for (int n = 0; n < TN / 16; ++n)
#pragma unroll
                        for (int m = 0; m < TM / 16; ++m)
                            acc[n][m] = mma(fw[n], fx[m], acc[n][m], sw[n], sx[m]);
                }
            }
            at = at + kStage == kLds ? 0 : at + kStage;
            next = next + kStage == kLds ? 0 : next + kStage;
        }
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

template <bool OUT_BF16, int BM, int BN, int WM, int WN, int STAGES>
hipError_t matmul_tiles(const ExpertShape &sh, const int32_t *seg_ptr, const ScaledArgs &a,
                        hipStream_t st) {
    typedef ScaledProduct<BM, BN, WM, WN, STAGES> P;
    const int64_t tm = most_tiles(sh, BM), tn = tiles_of(sh.n_out, BN);
    const bool stream = (int64_t)sh.R * sh.SK * sh.n_out * (OUT_BF16 ? 2 : 4) >= kStreamBytes;
    return in_order(sh.R, tm, tn, 8, sh.R % 8 == 0, [&](const Order &order, uint32_t at, dim3 grid) {
        hipLaunchKernelGGL((k_matmul_mx<P, OUT_BF16, BM, BN>), grid, dim3(P::kThreads), 0, st, sh,
                           seg_ptr, a, order, at, stream);
    });
}

template <bool OUT_BF16>
hipError_t matmul(const ExpertShape &sh, const int32_t *seg_ptr, const ScaledArgs &a, hipStream_t st) {
    const int64_t segs = sh.G + sh.B / 2 < sh.SK ? sh.G + sh.B / 2 : sh.SK;
    const int64_t rows = tiles_of(sh.SK, (int)segs);
    auto tiles = [&](int bm, int bn) { return sh.R * segs * tiles_of(rows, bm) * tiles_of(sh.n_out, bn); };
    if (sh.n_out > 128 && rows >= 192 && fills(tiles(256, 256)))
        return matmul_tiles<OUT_BF16, 256, 256, 2, 4, 2>(sh, seg_ptr, a, st);
    if (sh.n_out > 64 && rows >= 40 && tiles(128, 128) >= kFill)
        return matmul_tiles<OUT_BF16, 128, 128, 2, 2, 2>(sh, seg_ptr, a, st);
    if (rows <= 16) return matmul_tiles<OUT_BF16, 32, 64, 2, 2, 4>(sh, seg_ptr, a, st);
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
