// The experts' products for gfx950: what happens to the rows between dispatch and
// combine. Dispatch leaves each rank's S*K rows grouped by expert, so the product
// of a rank is one matrix product for each segment, with ragged row counts:
//
//   y[t] = x[t] W_seg            k_matmul; also the gradient of x, with the
//                                columns' roles exchanged and W read the other way
//   dW_seg = sum_t x[t]^T g[t]   k_wgrad
//   y[t,n] = s_t s_n sum_i q[t,i] W_q[n,i]    the 8-bit form
#include <type_traits>

#include "experts.h"
#include "rows.h"

namespace moonep {
namespace {

using namespace rows;

constexpr int kThreads = 256;
constexpr int BM = 64, BN = 64, BK = 16;

typedef uint16_t bf16_t;

__device__ __forceinline__ float to_f32(bf16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ int to_f32(int8_t v) { return v; }

__device__ __forceinline__ void store_out(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_out(bf16_t *p, float v) {
    *p = (bf16_t)(pack_bf16x2(v, 0.0f) & 0xffffu);
}

// Sum of v over lanes 0 .. l, in every lane l.
__device__ __forceinline__ int wave_scan(int v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int up = __shfl_up(v, d);
        if (lane_id() >= d) v += up;
    }
    return v;
}

struct Tile {
    int seg, row, rows;  // segment (-1: none), first row on the rank, rows
};

// Tile `want` of a rank whose segments are cut into tiles of at most `bm` rows.
// Offsets are clamped to the rank's rows, so no table leads out of the arrays;
// a segment whose end is not past its start is empty.
__device__ Tile find_tile(const int32_t *ptr, int n, int SK, int bm, int want) {
    int base = 0;
    for (int s = 0; s < n; s += 64) {
        const int j = s + lane_id();
        int lo = 0, len = 0;
        if (j < n) {
            lo = ptr[j];
            const int hi = min(ptr[j + 1], SK);
            len = lo >= 0 && hi > lo ? hi - lo : 0;
        }
        const int tiles = (len + bm - 1) / bm;
        const int upto = wave_scan(tiles);
        const int total = readlane_i(upto, 63);
        if (want < base + total) {
            const int l = __ffsll((unsigned long long)__ballot(base + upto > want)) - 1;
            const int first = (want - base - (readlane_i(upto, l) - readlane_i(tiles, l))) * bm;
            return {s + l, readlane_i(lo, l) + first, min(bm, readlane_i(len, l) - first)};
        }
        base += total;
    }
    return {-1, 0, 0};
}

// y tile = x rows * W columns, one 64x64 tile for each workgroup, 4x4 for each thread.
template <typename T, typename Out, bool TRANSPOSED>
__global__ __launch_bounds__(kThreads) void k_matmul(ExpertShape sh, const int32_t *seg_ptr,
                                                     const T *x, const float *x_scale, const T *w,
                                                     const float *w_scale, const T *dup_w,
                                                     const float *dup_scale, Out *y, int tiles_m,
                                                     int tiles_n, int64_t first) {
    using Acc = typename std::conditional<std::is_same<T, int8_t>::value, int, float>::type;
    __shared__ Acc s_x[BK][BM + 1], s_w[BK][BN + 1];
    const int64_t id = first + blockIdx.x;
    const int n0 = (int)(id % tiles_n) * BN;
    const int64_t rm = id / tiles_n;
    const int r = (int)(rm / tiles_m);
    const Tile t = find_tile(seg_ptr + (int64_t)r * (sh.n_seg + 1), sh.G + sh.B, sh.SK, BM,
                             (int)(rm % tiles_m));
    if (t.seg < 0) return;
    const bool home = t.seg < sh.G;
    const int64_t which = home ? (int64_t)r * sh.G + t.seg : (int64_t)r * sh.slots + t.seg - sh.G;
    const T *wm = (home ? w : dup_w) + which * sh.block;
    const int64_t row0 = (int64_t)r * sh.SK + t.row;
    const T *xm = x + row0 * sh.n_in;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    Acc acc[4][4] = {};
    for (int k0 = 0; k0 < sh.n_in; k0 += BK) {
        for (int i = threadIdx.x; i < BK * BM; i += kThreads) {
            const int k = i % BK, m = i / BK;
            s_x[k][m] = m < t.rows && k0 + k < sh.n_in ? to_f32(xm[(int64_t)m * sh.n_in + k0 + k])
                                                       : Acc(0);
        }
        for (int i = threadIdx.x; i < BK * BN; i += kThreads) {
            const int k = TRANSPOSED ? i % BK : i / BN, n = TRANSPOSED ? i / BK : i % BN;
            Acc v = 0;
            if (n0 + n < sh.n_out && k0 + k < sh.n_in)
                v = to_f32(TRANSPOSED ? wm[(int64_t)(n0 + n) * sh.n_in + k0 + k]
                                      : wm[(int64_t)(k0 + k) * sh.n_out + n0 + n]);
            s_w[k][n] = v;
        }
        __syncthreads();
        for (int k = 0; k < BK; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] += s_x[k][ty * 4 + i] * s_w[k][tx * 4 + j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int m = ty * 4 + i, n = n0 + tx * 4 + j;
            if (m >= t.rows || n >= sh.n_out) continue;
            float v = (float)acc[i][j];
            if constexpr (std::is_same<T, int8_t>::value)
                v = v * x_scale[row0 + m] * (home ? w_scale : dup_scale)[which * sh.scale_block + n];
            store_out(y + (row0 + m) * sh.n_out + n, v);
        }
}

// One 64x64 tile of a segment's weight gradient, over all of the segment's rows.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_wgrad(ExpertShape sh, const int32_t *seg_ptr,
                                                    const T *a, const T *b, float *home,
                                                    float *dup, int n_a, int n_b, int tiles_a,
                                                    int tiles_b, int64_t first) {
    __shared__ float s_a[BK][BM + 1], s_b[BK][BN + 1];
    const int64_t id = first + blockIdx.x;
    const int b0 = (int)(id % tiles_b) * BN, a0 = (int)(id / tiles_b % tiles_a) * BM;
    const int64_t rs = id / ((int64_t)tiles_a * tiles_b);
    const int r = (int)(rs / (sh.G + sh.B)), j = (int)(rs % (sh.G + sh.B));
    const int32_t *ptr = seg_ptr + (int64_t)r * (sh.n_seg + 1) + j;
    const int lo = ptr[0], end = ptr[1], hi = min(end, sh.SK);
    if (j >= sh.G && (lo < 0 || end < lo)) return;
    const int rows = lo >= 0 && hi > lo ? hi - lo : 0;
    float *out = j < sh.G ? home + ((int64_t)r * sh.G + j) * sh.block
                          : dup + ((int64_t)r * sh.slots + j - sh.G) * sh.block;
    const int64_t row0 = (int64_t)r * sh.SK + (rows > 0 ? lo : 0);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < rows; k0 += BK) {
        for (int i = threadIdx.x; i < BK * BM; i += kThreads) {
            const int k = i / BM, m = i % BM;
            const bool in = k0 + k < rows;
            s_a[k][m] = in && a0 + m < n_a ? to_f32(a[(row0 + k0 + k) * n_a + a0 + m]) : 0.0f;
            s_b[k][m] = in && b0 + m < n_b ? to_f32(b[(row0 + k0 + k) * n_b + b0 + m]) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < BK; ++k)
            for (int i = 0; i < 4; ++i)
                for (int c = 0; c < 4; ++c) acc[i][c] += s_a[k][ty * 4 + i] * s_b[k][tx * 4 + c];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int c = 0; c < 4; ++c) {
            const int m = a0 + ty * 4 + i, n = b0 + tx * 4 + c;
            if (m < n_a && n < n_b) out[(int64_t)m * n_b + n] = acc[i][c];
        }
}

// Rows to 8 bits, one wave for each row: the largest magnitude first, then the row again.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_quantize(int64_t n_rows, int cols, const T *x,
                                                       int8_t *q, float *scale) {
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64;
    if (row >= n_rows) return;
    const T *xr = x + row * cols;
    uint32_t most = 0;  // magnitudes compare like their bits, and a NaN's are the largest
    for (int c = lane_id(); c < cols; c += 64)
        most = max(most, __float_as_uint(to_f32(xr[c])) & 0x7fffffffu);
    for (int d = 32; d > 0; d /= 2) most = max(most, (uint32_t)__shfl_xor((int)most, d));
    const bool finite = most < 0x7f800000u;
    const float a = fmaxf(__uint_as_float(most), 0x1p-100f);
    const float inv = 127.0f / a;
    for (int c = lane_id(); c < cols; c += 64)
        q[row * cols + c] = finite ? (int8_t)(int)rintf(to_f32(xr[c]) * inv) : (int8_t)0;
    if (lane_id() == 0) scale[row] = finite ? a / 127.0f : __uint_as_float(0x7fc00000u);
}

// Launches `count` workgroups in pieces a grid can hold.
template <typename F>
hipError_t in_pieces(int64_t count, F &&launch) {
    constexpr int64_t kPiece = (int64_t)1 << 22;
    for (int64_t at = 0; at < count; at += kPiece) {
        launch(at, dim3((unsigned)(count - at < kPiece ? count - at : kPiece)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Most tiles of bm rows that the segments of one rank make.
int64_t most_tiles(const ExpertShape &sh, int bm) {
    const int64_t segs = sh.G + sh.B;
    return sh.SK / bm + (segs < sh.SK ? segs : sh.SK);
}

template <typename T, typename Out>
hipError_t matmul(const ExpertShape &sh, const int32_t *seg_ptr, const void *x, const float *xs,
                  const void *w, const float *ws, const void *dw, const float *ds, void *y,
                  hipStream_t st) {
    const int tm = (int)most_tiles(sh, BM), tn = (sh.n_out + BN - 1) / BN;
    return in_pieces((int64_t)sh.R * tm * tn, [&](int64_t at, dim3 grid) {
        if (sh.transposed)
            hipLaunchKernelGGL((k_matmul<T, Out, true>), grid, dim3(kThreads), 0, st, sh, seg_ptr,
                               (const T *)x, xs, (const T *)w, ws, (const T *)dw, ds, (Out *)y, tm, tn, at);
        else
            hipLaunchKernelGGL((k_matmul<T, Out, false>), grid, dim3(kThreads), 0, st, sh, seg_ptr,
                               (const T *)x, xs, (const T *)w, ws, (const T *)dw, ds, (Out *)y, tm, tn, at);
    });
}

template <typename T>
hipError_t wgrad(const ExpertShape &sh, const int32_t *seg_ptr, const void *x, const void *g,
                 float *home, float *dup, hipStream_t st) {
    // a gradient stored [n_out, n_in] is the product with its operands exchanged
    const void *a = sh.transposed ? g : x, *b = sh.transposed ? x : g;
    const int n_a = sh.transposed ? sh.n_out : sh.n_in, n_b = sh.transposed ? sh.n_in : sh.n_out;
    const int ta = (n_a + BM - 1) / BM, tb = (n_b + BN - 1) / BN;
    return in_pieces((int64_t)sh.R * (sh.G + sh.B) * ta * tb, [&](int64_t at, dim3 grid) {
        hipLaunchKernelGGL((k_wgrad<T>), grid, dim3(kThreads), 0, st, sh, seg_ptr, (const T *)a,
                           (const T *)b, home, dup, n_a, n_b, ta, tb, at);
    });
}

}  // namespace

hipError_t launch_expert_matmul(const ExpertShape &sh, const int32_t *seg_ptr, const void *x,
                                const void *w, const void *dup_w, void *y, int bf16,
                                hipStream_t st) {
    return bf16 ? matmul<bf16_t, bf16_t>(sh, seg_ptr, x, nullptr, w, nullptr, dup_w, nullptr, y, st)
                : matmul<float, float>(sh, seg_ptr, x, nullptr, w, nullptr, dup_w, nullptr, y, st);
}

hipError_t launch_expert_wgrad(const ExpertShape &sh, const int32_t *seg_ptr, const void *x,
                               const void *g, float *home, float *dup, int bf16, hipStream_t st) {
    return bf16 ? wgrad<bf16_t>(sh, seg_ptr, x, g, home, dup, st)
                : wgrad<float>(sh, seg_ptr, x, g, home, dup, st);
}

hipError_t launch_expert_matmul_quant(const ExpertShape &sh, const int32_t *seg_ptr,
                                      const int8_t *x, const float *x_scale, const int8_t *w,
                                      const float *w_scale, const int8_t *dup_w,
                                      const float *dup_scale, void *y, int y_bf16, hipStream_t st) {
    return y_bf16 ? matmul<int8_t, bf16_t>(sh, seg_ptr, x, x_scale, w, w_scale, dup_w, dup_scale, y, st)
                  : matmul<int8_t, float>(sh, seg_ptr, x, x_scale, w, w_scale, dup_w, dup_scale, y, st);
}

hipError_t launch_quantize_rows(int64_t n_rows, int32_t cols, const void *x, int bf16, int8_t *q,
                                float *scale, hipStream_t st) {
    const int64_t wgs = (n_rows + kThreads / 64 - 1) / (kThreads / 64);
    if (bf16)
        hipLaunchKernelGGL((k_quantize<bf16_t>), dim3((unsigned)wgs), dim3(kThreads), 0, st, n_rows,
                           cols, (const bf16_t *)x, q, scale);
    else
        hipLaunchKernelGGL((k_quantize<float>), dim3((unsigned)wgs), dim3(kThreads), 0, st, n_rows,
                           cols, (const float *)x, q, scale);
    return hipGetLastError();
}

}  // namespace moonep
