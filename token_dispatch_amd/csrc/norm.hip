// The root-mean-square norm of rows with the residual's addition, and its gradients, for
// gfx950.
//
//   h = x + residual        binary32, rounded to the rows' type (what sum_out holds)
//   inv = 1 / sqrt(sum h^2 / n + eps)     binary64, rounded to binary32
//   v = (h * inv) * gamma   binary32; out in the rows' type, in 8 bits or in 4
//
//   t = g * gamma
//   grad_x = inv (t - h inv (sum t h inv) / n)  (+ grad_sum)
//   grad_gamma = sum over rows of g (h inv)
//
// The squares are added in binary64: whatever order the lanes add in, inv is the same
// number but for one row in about 10^8, and what is rounded to 8 or 4 bits with it.
#include <type_traits>

#include "emit.h"
#include "layerops.h"

namespace moonep {
namespace {

using namespace emit;

template <bool BF16>
__device__ __forceinline__ v4u pack(const float *f) {
    if constexpr (BF16)
        return v4u{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7])};
    else
        return v4u{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                   __float_as_uint(f[3])};
}

template <bool BF16>
__device__ __forceinline__ v4u added(const v4u &x, const v4u &r) {
    constexpr int N = Chunk<BF16>::N;
    float a[N], b[N];
    Chunk<BF16>::unpack(x, a);
    Chunk<BF16>::unpack(r, b);
#pragma unroll
    for (int j = 0; j < N; ++j) a[j] += b[j];
    return pack<BF16>(a);
}

struct NormArgs {
    const v4u *x, *res, *gamma;
    v4u *sum;
    char *out, *scale;
    float *inv_rms;
    double eps;
    int64_t n_rows;
    int chunks;
    bool stream;
};

// LANES lanes hold a row in registers, CPL 16-byte chunks each; CPL = 0: rows too long for
// that, read again for each pass over them. Bound by HBM: 8192 rows of 7168 in bf16 with a
// residual (411 MB) take 80 us to 8 bits, 5.1 TB/s (6.2 to 6.8 in the rows' type at most lengths);
// loads past the caches' order took 85 to it. One such row takes 4.1 us, a chain of a load, a sum
// and a store. A row's chunks of sum_out and out are stored
// after the last read of the same chunks, so both may lie where x or the residual do.
template <bool BF16, int LANES, int CPL, int OUT>
__global__ __launch_bounds__(group_of(LANES)) void k_norm(NormArgs a, int64_t first) {
    constexpr int kThreads = group_of(LANES);
    constexpr int N = Chunk<BF16>::N, kRows = kThreads / LANES, R = CPL > 0 ? CPL : 1;
    __shared__ double ss_lds[kThreads / 64];
    __shared__ uint32_t most_lds[kThreads / 64];
    const int lane = threadIdx.x % LANES;
    const int64_t row = first + (int64_t)blockIdx.x * kRows + threadIdx.x / LANES;
    if (row >= a.n_rows) return;
    const int chunks = a.chunks;
    const v4u *x = a.x + row * chunks, *res = a.res ? a.res + row * chunks : nullptr;
    v4u h[R];
    double ss = 0;
    auto at = [&](int c) {
        const v4u q = x[c];
        return res ? added<BF16>(q, res[c]) : q;
    };
    auto square = [&](const v4u &q) {
        float f[N];
        Chunk<BF16>::unpack(q, f);
#pragma unroll
        for (int j = 0; j < N; ++j) ss = __builtin_fma((double)f[j], (double)f[j], ss);
    };
    if constexpr (CPL > 0) {
#pragma unroll
        for (int i = 0; i < CPL; ++i) {
            h[i] = v4u{0, 0, 0, 0};
            if (lane + i * LANES < chunks) h[i] = __builtin_nontemporal_load(x + lane + i * LANES);
        }
        if (res) {
            v4u r[R];
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
                r[i] = v4u{0, 0, 0, 0};
                if (lane + i * LANES < chunks) r[i] = __builtin_nontemporal_load(res + lane + i * LANES);
            }
#pragma unroll
            for (int i = 0; i < CPL; ++i) h[i] = added<BF16>(h[i], r[i]);
        }
#pragma unroll
        for (int i = 0; i < CPL; ++i) square(h[i]);
    } else {
        for (int c = lane; c < chunks; c += LANES) square(at(c));
    }
    ss = reduce<LANES>(ss, ss_lds, [](double p, double q) { return p + q; });
    const float inv = (float)(1.0 / sqrt(ss / (double)((int64_t)chunks * N) + a.eps));
    auto normed = [&](const v4u &q, int c, float *v) {
        float g[N];
        Chunk<BF16>::unpack(q, v);
        Chunk<BF16>::unpack(c < chunks ? a.gamma[c] : v4u{0, 0, 0, 0}, g);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = v[j] * inv * g[j];
    };
    Scale8 s = {};
    if constexpr (OUT == kInt8) {
        uint32_t most = 0;
        float v[N];
        if constexpr (CPL > 0) {
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
                normed(h[i], lane + i * LANES, v);
                most = max(most, magnitude<N>(v));
            }
        } else {
            for (int c = lane; c < chunks; c += LANES) {
                normed(at(c), c, v);
                most = max(most, magnitude<N>(v));
            }
        }
        s = scale8(reduce<LANES>(most, most_lds, [](uint32_t p, uint32_t q) { return max(p, q); }));
    }
    auto emit = [&](const v4u &q, int c) {
        float v[N];
        normed(q, c, v);
        if constexpr (OUT == kMx) {
            const int64_t cols = (int64_t)chunks * N;
            put4<N>(v, c, chunks, a.stream, reinterpret_cast<uint8_t *>(a.out) + row * (cols / 2),
                    reinterpret_cast<uint8_t *>(a.scale) + row * scale_pitch(cols));
        }
        if (c >= chunks) return;
        if constexpr (OUT == kSame)
            store_streamed(pack<BF16>(v), reinterpret_cast<v4u *>(a.out) + row * chunks + c, a.stream);
        if constexpr (OUT == kInt8)
            put8<N>(v, s, a.stream, reinterpret_cast<int8_t *>(a.out) + (row * chunks + c) * N);
        if (a.sum) store_streamed(q, a.sum + row * chunks + c, a.stream);
    };
    if constexpr (CPL > 0) {
#pragma unroll
        for (int i = 0; i < CPL; ++i) emit(h[i], lane + i * LANES);
    } else {
        // whole groups of lanes, so that the blocks' lanes are all there
        for (int c = lane; c - lane < chunks; c += LANES)
            emit(c < chunks ? at(c) : v4u{0, 0, 0, 0}, c);
    }
    if (lane == 0) {
        if constexpr (OUT == kInt8) reinterpret_cast<float *>(a.scale)[row] = s.scale;
        if (a.inv_rms) a.inv_rms[row] = inv;
    }
}

template <bool BF16, int LANES, int CPL, int OUT>
hipError_t norm_rows(const NormArgs &a, hipStream_t st) {
    constexpr int kThreads = group_of(LANES);
    constexpr int64_t kPiece = launch_groups(kThreads), kRows = kThreads / LANES;
    for (int64_t at = 0; at < a.n_rows; at += kPiece * kRows) {
        const int64_t wgs = (a.n_rows - at + kRows - 1) / kRows;
        hipLaunchKernelGGL((k_norm<BF16, LANES, CPL, OUT>), dim3((unsigned)(wgs < kPiece ? wgs : kPiece)),
                           dim3(kThreads), 0, st, a, at);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Lanes of a row and its chunks a lane, by the row's chunks: enough of it in registers that none
// is read twice, few lanes idle, and enough rows on their way. With a residual, 134 MB of x, us
// (64 bf16 columns, 8 chunks, are 8 x 1):
//   bf16, 64       8 x 1 78, 16 x 2 136       bf16, 4096  256 x 2 80, 64 x 8 122
//   bf16, 512      64 x 1 82, 64 x 2 87       bf16, 12288, to 8 bits  512 x 4 102, 1024 x 2 122,
//   bf16, 2048     64 x 4 96, 256 x 1 93                              256 x 8 145
//   f32, 4096      512 x 2 80, 256 x 4 89     f32, 7168   1024 x 2 84, 512 x 4 90, 256 x 8 225
// Of few rows of up to 256 chunks each takes a workgroup, 64 lanes otherwise: 256 of 2048 columns
// 3.7 against 5.1 us, 1024 of them 5.1 against 6.0, 4096 14.7 against 13.2.
template <bool BF16, int OUT>
hipError_t norm_of(const NormArgs &a, hipStream_t st) {
    const int n = a.chunks;
    if (n <= 8) return norm_rows<BF16, 8, 1, OUT>(a, st);
    if (n <= 16) return norm_rows<BF16, 16, 1, OUT>(a, st);
    if (n <= 32) return norm_rows<BF16, 16, 2, OUT>(a, st);
    if (n <= 64) return norm_rows<BF16, 64, 1, OUT>(a, st);
    if (n <= 128) return norm_rows<BF16, 64, 2, OUT>(a, st);
    if (n <= 256 && a.n_rows >= 2048) return norm_rows<BF16, 64, 4, OUT>(a, st);
    if (n <= 256) return norm_rows<BF16, 256, 1, OUT>(a, st);
    if (n <= 512) return norm_rows<BF16, 256, 2, OUT>(a, st);
    if (n <= 1024) return norm_rows<BF16, BF16 ? 256 : 512, BF16 ? 4 : 2, OUT>(a, st);
    if (n <= 2048) return norm_rows<BF16, BF16 ? 512 : 1024, BF16 ? 4 : 2, OUT>(a, st);
    if (n <= 4096) return norm_rows<BF16, 1024, 4, OUT>(a, st);
    return norm_rows<BF16, 1024, 0, OUT>(a, st);
}

// ------------------------------------------------------------------ gradients

struct GradArgs {
    const v4u *go, *gsum, *x, *gamma;
    const float *inv_rms;
    v4u *gx;
    float *partial;  // [workgroups][cols], or NULL: left to k_gamma
    int64_t n_rows;
    int chunks;
    bool stream;
};

// Rows dealt to groups of LANES lanes, each of which keeps its rows' part of grad_gamma in
// registers; the groups of a workgroup add theirs up at the end, in order. Bound by HBM: 32768
// rows of 2048 in bf16 with a residual's gradient (537 MB) take 85 us, 6.4 TB/s, and the sum of
// 512 parts 4.8; with 1024 workgroups or 256, and loads in the caches' order, it took 101 and more.
template <bool BF16, int LANES, int CPL>
__global__ __launch_bounds__(group_of(LANES)) void k_norm_backward(GradArgs a) {
    constexpr int kThreads = group_of(LANES);
    constexpr int N = Chunk<BF16>::N, kGroups = kThreads / LANES, R = CPL > 0 ? CPL : 1;
    __shared__ float lds[2][kThreads / 64];
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES, chunks = a.chunks;
    const float per = 1.0f / (float)((int64_t)chunks * N);
    v4u gamma[R];
    // A lane's sums are binary64, so that the number of rows does not show in them (in binary32
    // they took 0 to 4% less time, and 2^19 equal rows of 1028 were off by 1e-5). They stay in
    // registers or, where those run out or leave fewer waves, in shared memory.
    constexpr bool kInLds = CPL > 0 && LANES * R * N >= 8192;
    static_assert(!kInLds || kGroups == 1, "a workgroup's rows are one at a time");
    __shared__ double own[kInLds ? R * N : 1][kInLds ? LANES : 1];
    double acc[kInLds ? 1 : R * N];
    auto sum = [&](int at) -> double & {
        if constexpr (kInLds) return own[at][lane];
        else return acc[at];
    };
#pragma unroll
    for (int i = 0; i < R; ++i) {
        gamma[i] = v4u{0, 0, 0, 0};
        if (CPL > 0 && lane + i * LANES < chunks) gamma[i] = a.gamma[lane + i * LANES];
#pragma unroll
        for (int j = 0; j < N; ++j) sum(i * N + j) = 0;
    }
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * kGroups + group; row < a.n_rows;
         row += (int64_t)gridDim.x * kGroups, turn ^= 1) {
        const v4u *x = a.x + row * chunks, *go = a.go + row * chunks;
        const float inv = a.inv_rms[row];
        float dot = 0;
        auto add = [&](const v4u &qx, const v4u &qg, const v4u &qw) {
            float x[N], g[N], w[N];
            Chunk<BF16>::unpack(qx, x);
            Chunk<BF16>::unpack(qg, g);
            Chunk<BF16>::unpack(qw, w);
#pragma unroll
            for (int j = 0; j < N; ++j) dot = fmaf(g[j] * w[j], x[j], dot);
        };
        auto put = [&](const v4u &qx, const v4u &qg, const v4u &qw, const v4u &qs, float mean, int c) {
            float x[N], g[N], w[N], s[N];
            Chunk<BF16>::unpack(qx, x);
            Chunk<BF16>::unpack(qg, g);
            Chunk<BF16>::unpack(qw, w);
            Chunk<BF16>::unpack(qs, s);
#pragma unroll
            for (int j = 0; j < N; ++j) s[j] += inv * (g[j] * w[j] - x[j] * inv * mean);
            store_streamed(pack<BF16>(s), a.gx + row * chunks + c, a.stream);
        };
        if constexpr (CPL > 0) {
            v4u qx[R], qg[R], qs[R];
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
                const int c = lane + i * LANES;
                qx[i] = qg[i] = qs[i] = v4u{0, 0, 0, 0};
                if (c < chunks) {
                    qx[i] = __builtin_nontemporal_load(x + c);
                    qg[i] = __builtin_nontemporal_load(go + c);
                    if (a.gsum) qs[i] = __builtin_nontemporal_load(a.gsum + row * chunks + c);
                }
            }
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
                add(qx[i], qg[i], gamma[i]);
                float x[N], g[N];
                Chunk<BF16>::unpack(qx[i], x);
                Chunk<BF16>::unpack(qg[i], g);
#pragma unroll
                for (int j = 0; j < N; ++j) sum(i * N + j) += (double)(g[j] * (x[j] * inv));
            }
            dot = reduce<LANES>(dot, lds[turn], [](float p, float q) { return p + q; });
            const float mean = dot * inv * per;
#pragma unroll
            for (int i = 0; i < CPL; ++i)
                if (lane + i * LANES < chunks)
                    put(qx[i], qg[i], gamma[i], qs[i], mean, lane + i * LANES);
        } else {
            for (int c = lane; c < chunks; c += LANES) add(x[c], go[c], a.gamma[c]);
            dot = reduce<LANES>(dot, lds[turn], [](float p, float q) { return p + q; });
            const float mean = dot * inv * per;
            for (int c = lane; c < chunks; c += LANES)
                put(x[c], go[c], a.gamma[c], a.gsum ? a.gsum[row * chunks + c] : v4u{0, 0, 0, 0}, mean, c);
        }
    }
    if constexpr (CPL > 0) {
        if (a.partial == nullptr) return;
        __shared__ double sums[kGroups > 1 ? kGroups : 1][kGroups > 1 ? LANES * R * N : 1];
        float *out = a.partial + (int64_t)blockIdx.x * chunks * N;
        if constexpr (kGroups > 1) {
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < N; ++j) sums[group][(lane + i * LANES) * N + j] = sum(i * N + j);
            __syncthreads();
            for (int c = threadIdx.x; c < chunks * N; c += kThreads) {
                double t = sums[0][c];
#pragma unroll
                for (int g = 1; g < kGroups; ++g) t += sums[g][c];
                out[c] = (float)t;
            }
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (lane + i * LANES < chunks)
#pragma unroll
                    for (int j = 0; j < N; j += 4)
                        *reinterpret_cast<v4f *>(out + (lane + i * LANES) * N + j) =
                            v4f{(float)sum(i * N + j), (float)sum(i * N + j + 1),
                                (float)sum(i * N + j + 2), (float)sum(i * N + j + 3)};
        }
    }
}

// grad_gamma's part of rows blockIdx.y, + gridDim.y, ... for rows too long for a workgroup's
// registers, in binary64 too.
constexpr int kGammaThreads = 256;
template <bool BF16>
__global__ __launch_bounds__(kGammaThreads) void k_gamma(GradArgs a, float *partial) {
    constexpr int N = Chunk<BF16>::N;
    const int c = blockIdx.x * kGammaThreads + threadIdx.x;
    if (c >= a.chunks) return;
    double acc[N] = {};
    for (int64_t row = blockIdx.y; row < a.n_rows; row += gridDim.y) {
        float x[N], g[N];
        Chunk<BF16>::unpack(a.x[row * a.chunks + c], x);
        Chunk<BF16>::unpack(a.go[row * a.chunks + c], g);
        const float inv = a.inv_rms[row];
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += (double)(g[j] * (x[j] * inv));
    }
    float *out = partial + ((int64_t)blockIdx.y * a.chunks + c) * N;
#pragma unroll
    for (int j = 0; j < N; ++j) out[j] = (float)acc[j];
}

// grad_gamma = the sum of n partial rows: 64 columns a workgroup, 16 lanes of 16 bytes to a
// row, the rows dealt to 64 of those and the 64 sums added in order.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void k_gamma_sum(const float *partial, int n, int cols,
                                                           float *out) {
    __shared__ double sums[64][64];
    const int part = threadIdx.x / 16, lane = threadIdx.x % 16, col = blockIdx.x * 64 + lane * 4;
    double s[4] = {};
    if (col < cols)
        for (int i = part; i < n; i += 64) {
            const v4f v = *reinterpret_cast<const v4f *>(partial + (int64_t)i * cols + col);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] += (double)v[j];
        }
#pragma unroll
    for (int j = 0; j < 4; ++j) sums[part][lane * 4 + j] = s[j];
    __syncthreads();
    const int c = blockIdx.x * 64 + threadIdx.x;
    if (threadIdx.x < 64 && c < cols) {
        double t = sums[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < 64; ++i) t += sums[i][threadIdx.x];
        out[c] = (float)t;
    }
}

template <bool BF16, int LANES, int CPL>
hipError_t norm_backward(const GradArgs &a, float *work, float *grad_gamma, hipStream_t st) {
    constexpr int kThreads = group_of(LANES);
    constexpr int N = Chunk<BF16>::N, kGroups = kThreads / LANES;
    const int64_t most = (a.n_rows + kGroups - 1) / kGroups;
    const int wgs = (int)(most < MOONEP_NORM_GRAD_ROWS ? most : MOONEP_NORM_GRAD_ROWS);
    GradArgs b = a;
    b.partial = grad_gamma && CPL > 0 ? work : nullptr;
    hipError_t e = hipSuccess;
    if (CPL == 0 && grad_gamma && wgs > 0) {  // first: grad_x may be written where grad_out lies
        const int across = (a.chunks + kGammaThreads - 1) / kGammaThreads;
        hipLaunchKernelGGL((k_gamma<BF16>), dim3(across, wgs), dim3(kGammaThreads), 0, st, a, work);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (wgs > 0) {
        hipLaunchKernelGGL((k_norm_backward<BF16, LANES, CPL>), dim3(wgs), dim3(kThreads), 0, st, b);
        e = hipGetLastError();
    }
    if (e != hipSuccess || grad_gamma == nullptr) return e;
    const int cols = a.chunks * N;
    hipLaunchKernelGGL(k_gamma_sum, dim3((cols + 63) / 64), dim3(kSumThreads), 0, st, work, wgs,
                       cols, grad_gamma);
    return hipGetLastError();
}

// Lanes and chunks as for the norm. 134 MB of x with a residual's gradient, us with the sum:
// 64 bf16 columns 8 x 1 92, 64 x 1 476; 256 columns 16 x 2 90, 64 x 1 145; 2048 columns
// 64 x 4 87, 256 x 1 101; 4096 columns 256 x 2 91, 64 x 8 98; 12288 columns 1024 x 2 101,
// 512 x 4 105, 256 x 8 117 (106 with binary64 sums for the form that is taken, the others within 2%).
template <bool BF16>
hipError_t backward_of(const GradArgs &a, float *work, float *grad_gamma, hipStream_t st) {
    const int n = a.chunks;
    if (n <= 8) return norm_backward<BF16, 8, 1>(a, work, grad_gamma, st);
    if (n <= 16) return norm_backward<BF16, 16, 1>(a, work, grad_gamma, st);
    if (n <= 32) return norm_backward<BF16, 16, 2>(a, work, grad_gamma, st);
    if (n <= 64) return norm_backward<BF16, 64, 1>(a, work, grad_gamma, st);
    if (n <= 128) return norm_backward<BF16, 64, 2>(a, work, grad_gamma, st);
    if (n <= 256) return norm_backward<BF16, 64, 4>(a, work, grad_gamma, st);
    if (n <= 512) return norm_backward<BF16, 256, 2>(a, work, grad_gamma, st);
    if (n <= 1024) return norm_backward<BF16, 512, 2>(a, work, grad_gamma, st);
    if (n <= 2048) return norm_backward<BF16, 1024, 2>(a, work, grad_gamma, st);
    if constexpr (!BF16) {  // 64 sums a lane would not stay in registers
        if (n <= 4096) return norm_backward<BF16, 512, 8>(a, work, grad_gamma, st);
    }
    return norm_backward<BF16, 1024, 0>(a, work, grad_gamma, st);
}

}  // namespace

hipError_t launch_norm(const NormRows &n, hipStream_t st) {
    NormArgs a;
    a.x = static_cast<const v4u *>(n.x);
    a.res = static_cast<const v4u *>(n.residual);
    a.gamma = static_cast<const v4u *>(n.gamma);
    a.sum = static_cast<v4u *>(n.sum);
    a.out = static_cast<char *>(n.out);
    a.scale = static_cast<char *>(n.scale);
    a.inv_rms = n.inv_rms;
    a.eps = n.eps;
    a.n_rows = n.n_rows;
    a.chunks = n.cols / (n.bf16 ? 8 : 4);
    a.stream = n.n_rows * n.cols * (n.bf16 ? 2 : 4) >= kStreamBytes;
    switch (n.out_kind * 2 + n.bf16) {
        case kSame * 2: return norm_of<false, kSame>(a, st);
        case kSame * 2 + 1: return norm_of<true, kSame>(a, st);
        case kInt8 * 2: return norm_of<false, kInt8>(a, st);
        case kInt8 * 2 + 1: return norm_of<true, kInt8>(a, st);
        case kMx * 2: return norm_of<false, kMx>(a, st);
        default: return norm_of<true, kMx>(a, st);
    }
}

hipError_t launch_norm_backward(const NormGrad &n, hipStream_t st) {
    GradArgs a;
    a.go = static_cast<const v4u *>(n.grad_out);
    a.gsum = static_cast<const v4u *>(n.grad_sum);
    a.x = static_cast<const v4u *>(n.x);
    a.gamma = static_cast<const v4u *>(n.gamma);
    a.inv_rms = n.inv_rms;
    a.gx = static_cast<v4u *>(n.grad_x);
    a.partial = nullptr;
    a.n_rows = n.n_rows;
    a.chunks = n.cols / (n.bf16 ? 8 : 4);
    a.stream = n.n_rows * n.cols * (n.bf16 ? 2 : 4) >= kStreamBytes;
    return n.bf16 ? backward_of<true>(a, n.work, n.grad_gamma, st)
                  : backward_of<false>(a, n.work, n.grad_gamma, st);
}

}  // namespace moonep
