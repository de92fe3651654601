// The experts' gated activation and its gradients, for gfx950.
//
//   s = 1 / (1 + exp(-gate));  out = gate * s * up
//   grad_gate = grad_out * up * s (1 + gate (1 - s));  grad_up = grad_out * gate * s
//
// All of it in binary32; the result is rounded once, to the rows' type, to 8 bits with a
// scale for the row or to 4 bits with a scale for each block of 32. Bound by HBM: 131072 rows of
// 512 in bf16 (403 MB) take 59 us, 6.8 TB/s, and the gradients of 262144 rows of 1024 444. With
// expf and a division the arithmetic bound it where results are short: 61 us, and 135 in place of
// 98 for 130944 rows of 1024 to 4 bits.
#include <type_traits>

#include "emit.h"
#include "layerops.h"

namespace moonep {
namespace {

using namespace emit;

struct ActArgs {
    const v4u *gate, *up;
    char *out, *scale;
    int64_t n_rows, ld;  // ld: chunks from row to row of gate and up
    int chunks;
    bool stream;
};

template <int N>
__device__ __forceinline__ void gated(const float *g, const float *u, float *v) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = g[j] * sigmoid(g[j]) * u[j];
}

// LANES lanes to a row, a chunk each at a time. 8 bits need the row's largest value first:
// its values are kept in registers where CPL chunks a lane hold them, else made twice.
template <bool BF16, int LANES, int CPL, int OUT>
__global__ __launch_bounds__(group_of(LANES)) void k_swiglu(ActArgs a, int64_t first) {
    constexpr int kThreads = group_of(LANES);
    constexpr int N = Chunk<BF16>::N, kRows = kThreads / LANES, R = CPL > 0 ? CPL : 1;
    const int lane = threadIdx.x % LANES, chunks = a.chunks;
    const int64_t row = first + (int64_t)blockIdx.x * kRows + threadIdx.x / LANES;
    if (row >= a.n_rows) return;
    const v4u *gate = a.gate + row * a.ld, *up = a.up + row * a.ld;
    auto at = [&](int c, float *v) {
        float g[N], u[N];
        Chunk<BF16>::unpack(__builtin_nontemporal_load(gate + c), g);
        Chunk<BF16>::unpack(__builtin_nontemporal_load(up + c), u);
        gated<N>(g, u, v);
    };
    if constexpr (OUT == kInt8) {
        __shared__ uint32_t lds[kThreads / 64];
        float v[R][N] = {};
        uint32_t most = 0;
        if constexpr (CPL > 0) {
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
                if (lane + i * LANES < chunks) at(lane + i * LANES, v[i]);
                most = max(most, magnitude<N>(v[i]));
            }
        } else {
            for (int c = lane; c < chunks; c += LANES) {
                at(c, v[0]);
                most = max(most, magnitude<N>(v[0]));
            }
        }
        const Scale8 s = scale8(reduce<LANES>(most, lds, [](uint32_t p, uint32_t q) { return max(p, q); }));
        int8_t *q = reinterpret_cast<int8_t *>(a.out) + row * chunks * N;
        if constexpr (CPL > 0) {
#pragma unroll
            for (int i = 0; i < CPL; ++i)
                if (lane + i * LANES < chunks)
                    put8<N>(v[i], s, a.stream, q + (int64_t)(lane + i * LANES) * N);
        } else {
            for (int c = lane; c < chunks; c += LANES) {
                at(c, v[0]);
                put8<N>(v[0], s, a.stream, q + (int64_t)c * N);
            }
        }
        if (lane == 0) reinterpret_cast<float *>(a.scale)[row] = s.scale;
    } else {
        // whole groups of lanes, so that the blocks' lanes are all there
        for (int c = lane; c - lane < chunks; c += LANES) {
            float v[N] = {};
            if (c < chunks) at(c, v);
            if constexpr (OUT == kMx) {
                const int64_t cols = (int64_t)chunks * N;
                put4<N>(v, c, chunks, a.stream, reinterpret_cast<uint8_t *>(a.out) + row * (cols / 2),
                        reinterpret_cast<uint8_t *>(a.scale) + row * scale_pitch(cols));
            } else if (c < chunks) {
                const int64_t to = (row * chunks + c) * N;
                if (a.stream) store_elems<N, BF16, true>(a.out, to, v);
                else store_elems<N, BF16, false>(a.out, to, v);
            }
        }
    }
}

template <bool BF16, int LANES, int CPL, int OUT>
hipError_t swiglu_rows(const ActArgs &a, hipStream_t st) {
    constexpr int kThreads = group_of(LANES);
    constexpr int64_t kPiece = launch_groups(kThreads), kRows = kThreads / LANES;
    for (int64_t at = 0; at < a.n_rows; at += kPiece * kRows) {
        const int64_t wgs = (a.n_rows - at + kRows - 1) / kRows;
        hipLaunchKernelGGL((k_swiglu<BF16, LANES, CPL, OUT>), dim3((unsigned)(wgs < kPiece ? wgs : kPiece)),
                           dim3(kThreads), 0, st, a, at);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <bool BF16, int OUT>
hipError_t swiglu_of(const ActArgs &a, hipStream_t st) {
    const int n = a.chunks;
    if constexpr (OUT == kInt8) {
        // lanes of a row x its chunks a lane. 134 MB of each operand in bf16, us: 64 columns 8 x 1
        // 54, 16 x 2 101; 4096 columns 256 x 2 56, 64 x 8 64; 7168 columns 512 x 2 55, 256 x 4
        // 59, rows read twice 108
        if (n <= 8) return swiglu_rows<BF16, 8, 1, OUT>(a, st);
        if (n <= 32) return swiglu_rows<BF16, 16, 2, OUT>(a, st);
        if (n <= 128) return swiglu_rows<BF16, 64, 2, OUT>(a, st);
        if (n <= 256) return swiglu_rows<BF16, 64, 4, OUT>(a, st);
        if (n <= 512) return swiglu_rows<BF16, 256, 2, OUT>(a, st);
        if (n <= 1024) return swiglu_rows<BF16, 512, 2, OUT>(a, st);
        if (n <= 2048) return swiglu_rows<BF16, 1024, 2, OUT>(a, st);
        if (n <= 4096) return swiglu_rows<BF16, 1024, 4, OUT>(a, st);
        return swiglu_rows<BF16, 1024, 0, OUT>(a, st);
    } else {
        // 131072 rows of 512 in bf16: 59 us with 64 lanes, 60 with 128, 66 with 256; 130944 rows
        // of 1024 to 4 bits 96, 101, 124; 9362 rows of 7168 70 us with 64 lanes, 63 with 256, to
        // 4 bits 65 and 54; 1048576 rows of 64 71 us with 16 lanes, 60 with 8
        if (n <= 8) return swiglu_rows<BF16, 8, 0, OUT>(a, st);
        if (n <= 32) return swiglu_rows<BF16, 16, 0, OUT>(a, st);
        if (n <= 256) return swiglu_rows<BF16, 64, 0, OUT>(a, st);
        return swiglu_rows<BF16, 256, 0, OUT>(a, st);
    }
}

struct ActGradArgs {
    const v4u *go, *gate, *up;
    char *grad_gate, *grad_up;
    int64_t n_rows, ld, grad_ld;  // chunks from row to row
    int chunks;
    bool stream;
};

template <bool BF16, int LANES, int THREADS>
__global__ __launch_bounds__(THREADS) void k_swiglu_backward(ActGradArgs a, int64_t first) {
    constexpr int N = Chunk<BF16>::N, kRows = THREADS / LANES;
    const int64_t row = first + (int64_t)blockIdx.x * kRows + threadIdx.x / LANES;
    if (row >= a.n_rows) return;
    for (int c = threadIdx.x % LANES; c < a.chunks; c += LANES) {
        float g[N], u[N], go[N], dg[N], du[N];
        Chunk<BF16>::unpack(__builtin_nontemporal_load(a.gate + row * a.ld + c), g);
        Chunk<BF16>::unpack(__builtin_nontemporal_load(a.up + row * a.ld + c), u);
        Chunk<BF16>::unpack(__builtin_nontemporal_load(a.go + row * a.chunks + c), go);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float s = sigmoid(g[j]);
            dg[j] = go[j] * u[j] * s * (1.0f + g[j] * (1.0f - s));
            du[j] = go[j] * g[j] * s;
        }
        const int64_t to = (row * a.grad_ld + c) * N;
        if (a.stream) {
            store_elems<N, BF16, true>(a.grad_gate, to, dg);
            store_elems<N, BF16, true>(a.grad_up, to, du);
        } else {
            store_elems<N, BF16, false>(a.grad_gate, to, dg);
            store_elems<N, BF16, false>(a.grad_up, to, du);
        }
    }
}

template <bool BF16, int LANES, int THREADS>
hipError_t swiglu_backward_rows(const ActGradArgs &a, hipStream_t st) {
    constexpr int64_t kPiece = launch_groups(THREADS), kRows = THREADS / LANES;
    for (int64_t at = 0; at < a.n_rows; at += kPiece * kRows) {
        const int64_t wgs = (a.n_rows - at + kRows - 1) / kRows;
        hipLaunchKernelGGL((k_swiglu_backward<BF16, LANES, THREADS>),
                           dim3((unsigned)(wgs < kPiece ? wgs : kPiece)), dim3(THREADS), 0, st, a, at);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// A workgroup for each row: 262144 rows of 1024 bf16 values (2.7 GB) take 438 us, 6.1 TB/s, with
// 128 lanes to a row and a workgroup, 468 with two rows to a workgroup, 476 with four of 64.
template <bool BF16>
hipError_t swiglu_backward_of(const ActGradArgs &a, hipStream_t st) {
    if (a.chunks <= 8) return swiglu_backward_rows<BF16, 8, 256>(a, st);
    if (a.chunks <= 32) return swiglu_backward_rows<BF16, 16, 256>(a, st);
    if (a.chunks <= 64) return swiglu_backward_rows<BF16, 64, 64>(a, st);
    return swiglu_backward_rows<BF16, 128, 128>(a, st);
}

}  // namespace

hipError_t launch_swiglu(const GatedRows &g, hipStream_t st) {
    const int n = g.bf16 ? 8 : 4;
    ActArgs a;
    a.gate = static_cast<const v4u *>(g.gate);
    a.up = static_cast<const v4u *>(g.up);
    a.out = static_cast<char *>(g.out);
    a.scale = static_cast<char *>(g.scale);
    a.n_rows = g.n_rows;
    a.ld = g.ld / n;
    a.chunks = g.cols / n;
    a.stream = g.n_rows * g.cols * (g.bf16 ? 2 : 4) >= kStreamBytes;
    switch (g.out_kind * 2 + g.bf16) {
        case kSame * 2: return swiglu_of<false, kSame>(a, st);
        case kSame * 2 + 1: return swiglu_of<true, kSame>(a, st);
        case kInt8 * 2: return swiglu_of<false, kInt8>(a, st);
        case kInt8 * 2 + 1: return swiglu_of<true, kInt8>(a, st);
        case kMx * 2: return swiglu_of<false, kMx>(a, st);
        default: return swiglu_of<true, kMx>(a, st);
    }
}

hipError_t launch_swiglu_backward(const GatedGrad &g, hipStream_t st) {
    const int n = g.bf16 ? 8 : 4;
    ActGradArgs a;
    a.go = static_cast<const v4u *>(g.grad_out);
    a.gate = static_cast<const v4u *>(g.gate);
    a.up = static_cast<const v4u *>(g.up);
    a.grad_gate = static_cast<char *>(g.grad_gate);
    a.grad_up = static_cast<char *>(g.grad_up);
    a.n_rows = g.n_rows;
    a.ld = g.ld / n;
    a.grad_ld = g.grad_ld / n;
    a.chunks = g.cols / n;
    a.stream = g.n_rows * g.cols * (g.bf16 ? 2 : 4) >= kStreamBytes;
    return g.bf16 ? swiglu_backward_of<true>(a, st) : swiglu_backward_of<false>(a, st);
}

}  // namespace moonep
