// The experts' products for gfx950: what happens to the rows between dispatch and
// combine. Dispatch leaves each rank's S*K rows grouped by expert, so the product
// of a rank is one matrix product for each segment, with ragged row counts:
//
//   y[t] = x[t] W_seg            k_matmul; also the gradient of x, with the
//                                columns' roles exchanged and W read the other way
//   dW_seg = sum_t x[t]^T g[t]   k_wgrad
//   y[t,n] = s_t s_n sum_i q[t,i] W_q[n,i]    the 8-bit form
#include "emit.h"
#include "experts.h"
#include "rows.h"
#include "segments.h"
#include "tiles.h"

namespace moonep {
namespace {

using namespace rows;
using namespace segments;

constexpr int kThreads = 256;

// A tile of a segment's product. One launch makes the tiles of all segments: a workgroup finds
// its segment in the table itself, so no host reads the plan, and workgroups past a rank's last
// tile return at once. Long segments are bound by the loads and the matrix units together
// (262144 rows in 64 segments, 2048 -> 1024: 0.95 ms in bf16, 1.16 PFLOP/s; 0.55 ms in 8 bits, 2.0
// POP/s), short ones by their matrices' bytes (896 experts of 146 rows, 7168 -> 512: 1.81 ms, 4.7
// TB/s; 64 rows in all, 2048 -> 1024: 34 us, 6.0 TB/s; medians).
template <typename P, int EB, bool TRANSPOSED, bool OUT_BF16, int BM, int BN>
__global__ __launch_bounds__(P::kThreads) void k_matmul(ExpertShape sh, const int32_t *seg_ptr,
                                                        const char *x, const float *x_scale,
                                                        const char *w, const float *w_scale,
                                                        const char *dup_w, const float *dup_scale,
                                                        void *y, Order order, uint32_t first,
                                                        bool stream) {
    __shared__ __align__(1024) char lds[P::kLds];
    const Place at = place(order, first);
    if (at.unit < 0) return;
    const int r = at.unit;
    const Tile t = find_tile(seg_ptr + (int64_t)r * (sh.n_seg + 1), sh.G + sh.B, sh.SK, BM, at.m);
    if (t.seg < 0) return;
    const bool home = t.seg < sh.G;
    const int64_t which = home ? (int64_t)r * sh.G + t.seg : (int64_t)r * sh.slots + t.seg - sh.G;
    const char *wm = (home ? w : dup_w) + which * sh.block * EB;
    const int64_t row0 = (int64_t)r * sh.SK + t.row;
    const int n0 = at.n * BN;
    typename P::X px;
    typename P::W pw;
    px.init(x + row0 * sh.n_in * EB, sh.n_in * EB, t.rows, 0);
    if constexpr (TRANSPOSED)
        pw.init(wm + (int64_t)n0 * sh.n_in * EB, sh.n_in * EB, min(BN, sh.n_out - n0), 0);
    else
        pw.init(wm + n0 * EB, sh.n_out * EB, sh.n_in, n0 * EB);
    typename P::Sums acc;
    P::run(px, pw, sh.n_in, t.rows, lds, acc);
    if (!P::holds()) return;
    char *out = static_cast<char *>(y) + (row0 * sh.n_out + n0) * (OUT_BF16 ? 2 : 4);
    if constexpr (EB == 1) {
        const float *xs = x_scale + row0;
        const float *ws = (home ? w_scale : dup_scale) + which * sh.scale_block + n0;
        P::template put<OUT_BF16>(lds, acc, t.rows, sh.n_out - n0, out, sh.n_out, stream,
                                  [&](int row, int col, float *v) {
                                      const float s = xs[min(row, t.rows - 1)];
                                      // the last four columns in the place of those behind them
                                      const v4f c = *reinterpret_cast<const v4f *>(
                                          ws + min(col, sh.n_out - n0 - 4));
#pragma unroll
                                      for (int j = 0; j < 4; ++j) v[j] = v[j] * s * c[j];
                                  });
    } else {
        P::template put<OUT_BF16>(lds, acc, t.rows, sh.n_out - n0, out, sh.n_out, stream,
                                  [](int, int, float *) {});
    }
}

// A tile of a segment's weight gradient, over all of the segment's rows: the sums stay in
// registers from the first row to the last, so a gradient is written once and rows behind the
// segment (zeros by the range check) add nothing. Bound like the product above where segments are
// long (4096 rows on average: 0.95 ms, 1.16 PFLOP/s), by the gradients' own bytes where they are
// short (7168 x 512, skewed, 131072 rows in 116 segments: 1.06 ms, 3.5 TB/s of which 1.7 GB are
// written). Starting a rank's long segments first gains nothing there (1094 / 1095 us).
template <typename P, int EB, int BM, int BN>
__global__ __launch_bounds__(P::kThreads) void k_wgrad(ExpertShape sh, const int32_t *seg_ptr,
                                                       const char *a, const char *b, float *home,
                                                       float *dup, int n_a, int n_b, Order order,
                                                       uint32_t first, bool stream) {
    __shared__ __align__(1024) char lds[P::kLds];
    const Place at = place(order, first);
    if (at.unit < 0) return;
    const int r = at.unit / (sh.G + sh.B), j = at.unit - r * (sh.G + sh.B);
    const int32_t *ptr = seg_ptr + (int64_t)r * (sh.n_seg + 1) + j;
    const int lo = ptr[0], end = ptr[1], hi = min(end, sh.SK);
    if (j >= sh.G && (lo < 0 || end < lo)) return;
    const int rows = lo >= 0 && hi > lo ? hi - lo : 0;
    float *out = j < sh.G ? home + ((int64_t)r * sh.G + j) * sh.block
                          : dup + ((int64_t)r * sh.slots + j - sh.G) * sh.block;
    const int64_t row0 = (int64_t)r * sh.SK + (rows > 0 ? lo : 0);
    const int a0 = at.m * BM, b0 = at.n * BN;
    typename P::X pa;
    typename P::W pb;
    pa.init(a + (row0 * n_a + a0) * EB, n_a * EB, rows, a0 * EB);
    pb.init(b + (row0 * n_b + b0) * EB, n_b * EB, rows, b0 * EB);
    typename P::Sums acc;
    P::run(pa, pb, rows, n_a - a0, lds, acc);
    if (!P::holds()) return;
    P::template put<false>(lds, acc, n_a - a0, n_b - b0, out + (int64_t)a0 * n_b + b0, n_b,
                           stream, [](int, int, float *) {});
}

// Rows to 8 bits: LANES lanes hold a row in registers, CPL 16-byte chunks each, so a row
// is read once. Bound by HBM: 3 bytes an element from bf16 (131072 rows of 7168: 2.8 GB in 0.46
// ms, 6.2 TB/s). From binary32 it is not: 262144 rows of 2048 take 0.92 ms, 2.9 TB/s, with and
// without the stores past the caches; a wave stores 256 bytes at a time there.
//
// The largest magnitude is found on the bits without the sign, two values of a word at a time in
// bf16; the scale and the codes are made as everywhere (emit.h).
template <bool BF16>
__device__ __forceinline__ uint32_t magnitude(const v4u &q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (BF16) most = max(max(most, w[j] << 16 & 0x7fff0000u), w[j] & 0x7fff0000u);
        else most = max(most, w[j] & 0x7fffffffu);
    }
    return most;
}

template <bool BF16>
__device__ __forceinline__ void put_quantized(const v4u &q, const emit::Scale8 &s, bool stream,
                                              int8_t *to) {
    constexpr int N = rows::Chunk<BF16>::N;
    float x[N];
    rows::Chunk<BF16>::unpack(q, x);
    emit::put8<N>(x, s, stream, to);
}

// CPL = 0: rows too long for registers, read twice.
template <bool BF16, int LANES, int CPL>
__global__ __launch_bounds__(kThreads) void k_quantize(int64_t first, int64_t n_rows, int chunks,
                                                       const v4u *__restrict__ x,
                                                       int8_t *__restrict__ q,
                                                       float *__restrict__ scale, bool stream) {
    constexpr int N = rows::Chunk<BF16>::N, kRows = kThreads / LANES, R = CPL > 0 ? CPL : 1;
    const int lane = threadIdx.x % LANES;
    const int64_t row = first + (int64_t)blockIdx.x * kRows + threadIdx.x / LANES;
    if (row >= n_rows) return;
    const v4u *xr = x + row * chunks;
    int8_t *qr = q + row * chunks * N;
    v4u v[R];
    uint32_t most = 0;
    if constexpr (CPL > 0) {
#pragma unroll
        for (int i = 0; i < CPL; ++i) {
            v[i] = v4u{0, 0, 0, 0};
            if (lane + i * LANES < chunks) v[i] = __builtin_nontemporal_load(xr + lane + i * LANES);
        }
#pragma unroll
        for (int i = 0; i < CPL; ++i) most = max(most, magnitude<BF16>(v[i]));
    } else {
        for (int c = lane; c < chunks; c += LANES) most = max(most, magnitude<BF16>(xr[c]));
    }
#pragma unroll
    for (int d = LANES / 2; d > 0; d /= 2) most = max(most, (uint32_t)__shfl_xor((int)most, d));
    const emit::Scale8 s = emit::scale8(most);
    if constexpr (CPL > 0) {
#pragma unroll
        for (int i = 0; i < CPL; ++i) {
            const int c = lane + i * LANES;
            if (c < chunks) put_quantized<BF16>(v[i], s, stream, qr + (int64_t)c * N);
        }
    } else {
        for (int c = lane; c < chunks; c += LANES)
            put_quantized<BF16>(xr[c], s, stream, qr + (int64_t)c * N);
    }
    if (lane == 0) scale[row] = s.scale;
}

template <bool BF16, int LANES, int CPL>
hipError_t quantize_rows(int64_t n_rows, int chunks, const void *x, int8_t *q, float *scale,
                         hipStream_t st) {
    constexpr int64_t kPiece = (int64_t)1 << 22, kRows = kThreads / LANES;
    const bool stream = n_rows * chunks * rows::Chunk<BF16>::N >= kStreamBytes;
    for (int64_t at = 0; at < n_rows; at += kPiece * kRows) {
        const int64_t wgs = (n_rows - at + kRows - 1) / kRows;
        hipLaunchKernelGGL((k_quantize<BF16, LANES, CPL>), dim3((unsigned)(wgs < kPiece ? wgs : kPiece)),
                           dim3(kThreads), 0, st, at, n_rows, chunks, static_cast<const v4u *>(x), q,
                           scale, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// A quarter of a wave for rows of up to 32 chunks (of 16 bytes), a wave for longer ones, with as few
// registers as hold the row; read twice where 16 chunks a lane do not. 1 GB of bf16, us, the
// variant taken against the next one:
//   chunks     32        64        128       256       512       896
//            248/525   306/339   240/244   250/244   246/244   252/383 (read twice)
template <bool BF16>
hipError_t quantize(int64_t n_rows, int chunks, const void *x, int8_t *q, float *scale,
                    hipStream_t st) {
    if (chunks <= 32) return quantize_rows<BF16, 16, 2>(n_rows, chunks, x, q, scale, st);
    if (chunks <= 128) return quantize_rows<BF16, 64, 2>(n_rows, chunks, x, q, scale, st);
    if (chunks <= 256) return quantize_rows<BF16, 64, 4>(n_rows, chunks, x, q, scale, st);
    if (chunks <= 512) return quantize_rows<BF16, 64, 8>(n_rows, chunks, x, q, scale, st);
    if (chunks <= 1024) return quantize_rows<BF16, 64, 16>(n_rows, chunks, x, q, scale, st);
    return quantize_rows<BF16, 64, 0>(n_rows, chunks, x, q, scale, st);
}

struct Operands {
    const int32_t *seg_ptr;
    const void *x;
    const float *x_scale;
    const void *w;
    const float *w_scale;
    const void *dup_w;
    const float *dup_scale;
    void *y;
};

template <int EB, bool TRANSPOSED, bool OUT_BF16, int BM, int BN, int WM, int WN, int WK,
          int STAGES, int KB = 128, bool PIPED = false>
hipError_t matmul_tiles(const ExpertShape &sh, const Operands &o, hipStream_t st) {
    typedef tiles::Product<EB, false, !TRANSPOSED, BM, BN, WM, WN, WK, STAGES, KB, PIPED> P;
    const int64_t tm = most_tiles(sh, BM), tn = tiles_of(sh.n_out, BN);
    const bool stream = (int64_t)sh.R * sh.SK * sh.n_out * (OUT_BF16 ? 2 : 4) >= kStreamBytes;
    return in_order(sh.R, tm, tn, 8, sh.R % 8 == 0, [&](const Order &order, uint32_t at, dim3 grid) {
        hipLaunchKernelGGL((k_matmul<P, EB, TRANSPOSED, OUT_BF16, BM, BN>), grid, dim3(P::kThreads), 0,
                           st, sh, o.seg_ptr, (const char *)o.x, o.x_scale, (const char *)o.w,
                           o.w_scale, (const char *)o.dup_w, o.dup_scale, o.y, order, at, stream);
    });
}

// The tile is chosen by the rows that a segment has on average (half the duplicate slots
// counted as used) and the tiles that makes. Measured with 256 segments of 0.3 to 1.7 times
// the rows, us in bf16, 2048 -> 1024 columns from [in, out] / [out, in] matrices:
//   rows        32x64     64x64     128x128    128x256    256x256
//      4      188/183   189/182
//     16      198/194   205/204    192/187    186/187
//     32      232/230   213/200    213/214    202/209
//     40      253/254   244/238    203/197    195/198
//    128                           293/292    263/266    240/254
//    160                           326/317    299/295    306/317
//    224                           397/389    370/373    330/344
//    500                                                 616/580
// 128x256 and 256x256 change places between 96 and 192 rows as segments come to pass 256; with
// the routing of a skewed layer, half of whose segments are short, they are equal at 128 in
// bf16, and in 8 bits 128x256 is 3% faster there. 128x128, two workgroups of which share a
// compute unit, hides more of the stores, which counts for few steps (128 segments of 512
// rows, 2048 columns out, 128x128 / 128x256 / 256x256):
//   columns in        128            256            512            1024
//   bf16          97/111/105    125/144/131    228/224/199    390/376/331
//   8 bits        95/100/99     108/119/112    142/151/134    250/240/208
// Too few tiles: the next smaller ones, and at last the waves of a workgroup share the steps,
// if each has one at least (2 rows 7168 -> 512: 9 us against 33 to 37 with 64x64). Two tiles a
// compute unit or fewer leave room for a third stage of 64x64 (32 segments of 64 rows, 2048 ->
// 256: 17.5 to 12.5 us; 21 of 238 rows, 264 -> 520, where more tiles could share a unit: 9.8 to
// 10.6). In f32 a tile of 32x64 loses nothing to 64x64, the matrix units being 10 times slower,
// and leaves fewer rows empty (128 segments of 256 rows, 2048 -> 1024: 1148 / 1206 us, of 64 rows
// 375 / 419, 16 of 4 rows, 4096 -> 2048: 138 / 156; 128x128 1250, 503, -).
template <int EB, bool TRANSPOSED, bool OUT_BF16>
hipError_t matmul(const ExpertShape &sh, const Operands &o, hipStream_t st) {
    const int64_t segs = sh.G + sh.B / 2 < sh.SK ? sh.G + sh.B / 2 : sh.SK;
    const int64_t rows = tiles_of(sh.SK, (int)segs);
    auto tiles = [&](int bm, int bn) { return sh.R * segs * tiles_of(rows, bm) * tiles_of(sh.n_out, bn); };
    if constexpr (EB != 4) {
        const int64_t step = (int64_t)sh.n_in * EB;
        if (sh.n_out > 128 && step > 512 && rows >= (EB == 1 ? 192 : 96) && fills(tiles(256, 256)))
            return matmul_tiles<EB, TRANSPOSED, OUT_BF16, 256, 256, 2, 4, 1, 5, 128, true>(sh, o, st);
        const int few = TRANSPOSED ? 40 : 16;
        if (sh.n_out > 128 && step > 1024 && rows >= few && fills(tiles(128, 256)))
            return matmul_tiles<EB, TRANSPOSED, OUT_BF16, 128, 256, 2, 4, 1, 3>(sh, o, st);
        if (sh.n_out > 64 && rows >= few && tiles(128, 128) >= kFill)
            return matmul_tiles<EB, TRANSPOSED, OUT_BF16, 128, 128, 2, 2, 1, 2>(sh, o, st);
    }
    if (tiles(64, 64) >= kFill || (int64_t)sh.n_in * EB < 8 * 128) {
        if constexpr (EB == 4) {
            return matmul_tiles<EB, TRANSPOSED, OUT_BF16, 32, 64, 2, 2, 1, 2>(sh, o, st);
        } else {
            if (rows <= 16) return matmul_tiles<EB, TRANSPOSED, OUT_BF16, 32, 64, 2, 2, 1, 4>(sh, o, st);
            if (tiles(64, 64) < 2 * kCus)
                return matmul_tiles<EB, TRANSPOSED, OUT_BF16, 64, 64, 2, 2, 1, 3>(sh, o, st);
            return matmul_tiles<EB, TRANSPOSED, OUT_BF16, 64, 64, 2, 2, 1, 2>(sh, o, st);
        }
    }
    if constexpr (EB != 4)
        if (rows <= 16) return matmul_tiles<EB, TRANSPOSED, OUT_BF16, 16, 32, 1, 1, 8, 2>(sh, o, st);
    return matmul_tiles<EB, TRANSPOSED, OUT_BF16, 32, 32, 1, 1, 8, 2>(sh, o, st);
}

template <int EB, int BM, int BN, int WM, int WN, int WK, int STAGES, int KB = 128,
          bool PIPED = false>
hipError_t wgrad_tiles(const ExpertShape &sh, const int32_t *seg_ptr, const void *x, const void *g,
                       float *home, float *dup, hipStream_t st) {
    typedef tiles::Product<EB, true, true, BM, BN, WM, WN, WK, STAGES, KB, PIPED> P;
    // a gradient stored [n_out, n_in] is the product with its operands exchanged
    const void *a = sh.transposed ? g : x, *b = sh.transposed ? x : g;
    const int n_a = sh.transposed ? sh.n_out : sh.n_in, n_b = sh.transposed ? sh.n_in : sh.n_out;
    const int64_t ta = tiles_of(n_a, BM), tb = tiles_of(n_b, BN);
    const bool stream = (int64_t)sh.R * sh.G * n_a * n_b * 4 >= kStreamBytes;
    // whole ranks of segments have equal work; else the segments are dealt out
    const int64_t segs = (int64_t)sh.R * (sh.G + sh.B);
    return in_order(segs, ta, tb, 4, sh.R % 8 == 0, [&](const Order &order, uint32_t at, dim3 grid) {
        hipLaunchKernelGGL((k_wgrad<P, EB, BM, BN>), grid, dim3(P::kThreads), 0, st, sh, seg_ptr,
                           (const char *)a, (const char *)b, home, dup, n_a, n_b, order, at, stream);
    });
}

// Measured in bf16 with segments of 0.3 to 1.7 times the rows, us:
//                                64x64   64x64/4   128x128   256x256     /4: four waves share
//   128 x 64 rows   1024x1024     110               99        105            the steps
//   128 x 128 rows  1024x1024     130               117       113
//   128 x 256 rows  1024x1024     175               153       137
//   16 x 1024 rows  1024x512      33      65        30        42
//   128 x 4096 rows 256x256       197     210       157       172
//   64 x 4096 rows  256x256       101     101       109       157
//   32 x 4096 rows  256x256       56      40        102       155
//   4 x 8192 rows   512x512       82      47        145       223
//   4 x 256 rows    512x512       5.7     7.7       10        16
// and 32x32/4 against 64x64 where few tiles have many steps: 4 x 512 rows of 256x256 4.8 / 6.0,
// 8 x 512 rows 6.1 / 6.0, 4 x 128 rows 4.0 / 4.0.
//
// In f32, whose products are 10 times slower, smaller tiles spread better. Measured over 1355
// shapes: 1 to 128 segments of 16 to 4096 rows, 14 sizes from 128x128 to 2056x264; rows and tiles as
// the rule counts them, geometric means. 64x64 by eight waves over 32x32 by four, by the tiles of
// 64x64:
//                                  512    768    1024   1536   2048   4096   8192 and more
//   every 64x64 full               0.97   0.93   0.92   0.92   0.91   0.84   0.81
//   3 to 13% more than 32x32 need  1.08   1.05   1.06   0.96   0.88   0.80   0.83
//   13 to 44% more                 1.18   1.21   1.12   1.05   1.01   0.91   0.90
// so 64x64 from 6 tiles a unit on. 32x32/4 over the better of these two, by rows / tiles of 32x32:
//     1/16    1/8     1/4     1/2     1       2       4
//     1.28    1.17    1.06    0.96    0.90    0.85    0.78
// and from 1/4 on: between 1/4 and 1/2 the others are 6% faster on average and 35% at most, but 66%
// slower where the longest of a few segments sets the time (32 x 2048 rows, 264x520: 217 / 362 us).
// With these borders the rule's form is 2.9% above the fastest of the three on average, 35% at
// most; borders from 512 to 4096 tiles and from 1/4 to 1/2, by how full the tiles are too, gain 0.8%
// at most, and those with 1/2 lose 66% somewhere.
template <int EB>
hipError_t wgrad(const ExpertShape &sh, const int32_t *seg_ptr, const void *x, const void *g,
                 float *home, float *dup, hipStream_t st) {
    const int64_t segs = sh.G + sh.B / 2 < sh.SK ? sh.G + sh.B / 2 : sh.SK;
    const int64_t rows = sh.SK / segs;
    auto tiles = [&](int b) { return sh.R * segs * tiles_of(sh.n_in, b) * tiles_of(sh.n_out, b); };
    if constexpr (EB != 4) {
        const int least = sh.n_in < sh.n_out ? sh.n_in : sh.n_out;
        if (least > 128 && rows >= 128 && tiles(256) >= kFill)
            return wgrad_tiles<EB, 256, 256, 2, 4, 1, 8, 64, true>(sh, seg_ptr, x, g, home, dup, st);
        if (least > 64 && tiles(128) >= 2 * kFill)
            return wgrad_tiles<EB, 128, 128, 2, 2, 1, 2>(sh, seg_ptr, x, g, home, dup, st);
        if (rows >= 1024 && tiles(64) >= kFill / 2 && tiles(64) < 4 * kFill)
            return wgrad_tiles<EB, 64, 64, 1, 1, 4, 2>(sh, seg_ptr, x, g, home, dup, st);
    }
    if (EB == 4 ? 4 * rows >= tiles(32) : rows >= 256 && tiles(64) < kFill / 2)
        return wgrad_tiles<EB, 32, 32, 1, 1, 4, 2>(sh, seg_ptr, x, g, home, dup, st);
    if constexpr (EB == 4) {
        if (tiles(64) < 6 * kCus)
            return wgrad_tiles<EB, 32, 32, 2, 2, 1, 2>(sh, seg_ptr, x, g, home, dup, st);
        return wgrad_tiles<EB, 64, 64, 4, 2, 1, 2>(sh, seg_ptr, x, g, home, dup, st);
    } else {
        return wgrad_tiles<EB, 64, 64, 2, 2, 1, 2>(sh, seg_ptr, x, g, home, dup, st);
    }
}

}  // namespace

hipError_t launch_expert_matmul(const ExpertShape &sh, const int32_t *seg_ptr, const void *x,
                                const void *w, const void *dup_w, void *y, int bf16,
                                hipStream_t st) {
    const Operands o = {seg_ptr, x, nullptr, w, nullptr, dup_w, nullptr, y};
    if (bf16) return sh.transposed ? matmul<2, true, true>(sh, o, st) : matmul<2, false, true>(sh, o, st);
    return sh.transposed ? matmul<4, true, false>(sh, o, st) : matmul<4, false, false>(sh, o, st);
}

hipError_t launch_expert_wgrad(const ExpertShape &sh, const int32_t *seg_ptr, const void *x,
                               const void *g, float *home, float *dup, int bf16, hipStream_t st) {
    return bf16 ? wgrad<2>(sh, seg_ptr, x, g, home, dup, st)
                : wgrad<4>(sh, seg_ptr, x, g, home, dup, st);
}

hipError_t launch_expert_matmul_quant(const ExpertShape &sh, const int32_t *seg_ptr,
                                      const int8_t *x, const float *x_scale, const int8_t *w,
                                      const float *w_scale, const int8_t *dup_w,
                                      const float *dup_scale, void *y, int y_bf16, hipStream_t st) {
    const Operands o = {seg_ptr, x, x_scale, w, w_scale, dup_w, dup_scale, y};
    return y_bf16 ? matmul<1, true, true>(sh, o, st) : matmul<1, true, false>(sh, o, st);
}

hipError_t launch_quantize_rows(int64_t n_rows, int32_t cols, const void *x, int bf16, int8_t *q,
                                float *scale, hipStream_t st) {
    return bf16 ? quantize<true>(n_rows, cols / 8, x, q, scale, st)
                : quantize<false>(n_rows, cols / 4, x, q, scale, st);
}

}  // namespace moonep
