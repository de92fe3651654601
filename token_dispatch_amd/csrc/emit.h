// Values of a row from registers to memory: in the rows' type, in 8 bits with a scale for
// the row, or in 4 bits with a scale for each block of 32, for the kernels that make rows
// (norm.hip, activation.hip) or only quantise them (experts.hip, mx.hip), and the activation's
// sigmoid. Not part of the ABI.
#pragma once

#include "experts.h"
#include "rows.h"

namespace moonep {
namespace emit {

// Threads of a workgroup whose rows have LANES lanes each.
constexpr int group_of(int lanes) { return lanes > 256 ? lanes : 256; }

// Workgroups of one launch of rows: HIP refuses grids of 2^32 threads, which 2^22 workgroups of
// 1024 are.
constexpr int64_t launch_groups(int threads) {
    return ((int64_t)1 << 30) / threads < (int64_t)1 << 22 ? ((int64_t)1 << 30) / threads : (int64_t)1 << 22;
}

// Sum (or largest) of LANES lanes, in all of them; `lds` is used where they are a workgroup.
template <int LANES, typename T, typename F>
__device__ __forceinline__ T reduce(T v, T *lds, F &&f) {
#pragma unroll
    for (int d = (LANES < 64 ? LANES : 64) / 2; d > 0; d /= 2) v = f(v, __shfl_xor(v, d));
    if constexpr (LANES > 64) {
        if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
        __syncthreads();
        v = lds[0];
#pragma unroll
        for (int w = 1; w < LANES / 64; ++w) v = f(v, lds[w]);
    }
    return v;
}

using namespace rows;

enum Out { kSame, kInt8, kMx };

// Magnitudes are compared on the bits without the sign, which order like the magnitudes do
// and put infinity and then NaN above all numbers: one maximum tells finite rows from others.
constexpr uint32_t kInfBits = 0x7f800000u;

template <int N>
__device__ __forceinline__ uint32_t magnitude(const float *v) {
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) most = max(most, __float_as_uint(v[j]) & 0x7fffffffu);
    return most;
}

// The value of lane (this lane ^ D) for D = 1, 2 and, once all lanes of a quad have equal
// values, 4: moves within a row of 16 lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true));
}

// ------------------------------------------------------------------ activation

// 1 / (1 + exp(-g)), within 5 halves of a step, as the library's exponential and a division would
// have it: exp(-g) = 2^-m 2^f with m the integer nearest to g log2(e) and f what is left, by two
// parts of log2(e) (off by 2^-25 at most), so it is 2^m / (2^m + 2^f). The hardware's 2^f is off
// by a step, the sum by half a step, its reciprocal by half a step after a step of Newton's. No
// power passes the normal numbers, only the result may. Past 30 the sum is 2^m, from -104 down
// the result is zero.
__device__ __forceinline__ float sigmoid(float g) {
    const float x = __builtin_amdgcn_fmed3f(g, -104.0f, 30.0f);
    const float m = __builtin_rintf(x * 0x1.715476p+0f);
    const float f = fmaf(x, -0x1.4ae0cp-26f, fmaf(x, -0x1.715476p+0f, m));
    const float d = ldexpf(1.0f, (int)m) + __builtin_amdgcn_exp2f(f);
    const float r = __builtin_amdgcn_rcpf(d);
    return ldexpf(fmaf(r, fmaf(-d, r, 1.0f), r), (int)m);
}

// ------------------------------------------------------------------ 8 bits

struct Scale8 {
    float inv, scale;
    bool finite;
};

__device__ __forceinline__ Scale8 scale8(uint32_t most) {
    const bool finite = most < kInfBits;
    const float a = fmaxf(__uint_as_float(most), 0x1p-100f);
    return {finite ? 127.0f / a : 0.0f, finite ? a / 127.0f : __uint_as_float(0x7fc00000u), finite};
}

// A product of at most 127.00002 in magnitude goes to its nearest integer (ties to even) when
// 1.5 * 2^23 is added: the sum's last bit is worth 1, and its low byte is that integer.
template <int N>
__device__ __forceinline__ void put8(const float *v, const Scale8 &s, bool stream, int8_t *to) {
    uint32_t b[N], out[N / 4];
#pragma unroll
    for (int j = 0; j < N; ++j) {
#pragma clang fp contract(off)  // the product is rounded before it is added to
        const float p = v[j] * s.inv;
        b[j] = __float_as_uint(p + 12582912.0f);
    }
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
        const uint32_t lo = __builtin_amdgcn_perm(b[4 * j + 1], b[4 * j], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[4 * j + 3], b[4 * j + 2], 0x04000c0cu);
        out[j] = s.finite ? lo | hi : 0u;
    }
    typedef typename std::conditional<N == 8, v2u, uint32_t>::type V;
    V packed;
    __builtin_memcpy(&packed, out, sizeof(packed));
    store_streamed(packed, reinterpret_cast<V *>(to), stream);
}

// ------------------------------------------------------------------ 4 bits

// Bytes of a row's block scales: whole words, so that a word load never leaves the row.
__host__ __device__ inline int scale_pitch(int64_t cols) { return (int)((cols / 32 + 3) / 4 * 4); }

// N values of a block of 32, whose other values the 32 / N - 1 lanes beside this one hold
// (all of them active), at chunk c of the row.
//
// The scale is 2^(e - 127): e - 127 is two less than the exponent of the block's largest
// magnitude (6 = 1.5 * 2^2 is the largest code), rounded up from 1.75 of a power of two on:
// up to 1.75 * 4 = 7 the nearest code is 6, past it the doubled scale has a nearer one, so
// every value ends within half a step of codes. The value is scaled by a power of two, which
// is exact, and the conversion rounds to nearest even. A block with an infinity or a NaN gets
// e = 255, which stands for NaN, and codes of zero.
template <int N>
__device__ __forceinline__ void put4(const float *v, int c, int chunks, bool stream, uint8_t *q,
                                     uint8_t *scale) {
    uint32_t most = dpp_max<0x4e>(dpp_max<0xb1>(magnitude<N>(v)));  // quad_perm: lanes ^ 1, ^ 2
    if constexpr (N == 4) most = dpp_max<0x141>(most);              // row_half_mirror
    const bool finite = most < kInfBits;
    const int e = max((int)((most + 0x200000u) >> 23) - 2, 0);
    const float inv = finite ? __uint_as_float((uint32_t)(254 - e) << 23) : 0.0f;
    uint32_t codes = 0;
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        const float a = v[j] * inv, b = v[j + 1] * inv;
        if (j == 0) codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, a, b, 1.0f, 0);
        if (j == 2) codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, a, b, 1.0f, 1);
        if (j == 4) codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, a, b, 1.0f, 2);
        if (j == 6) codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, a, b, 1.0f, 3);
    }
    if (!finite) codes = 0;
    if (c >= chunks) return;
    if constexpr (N == 8)
        store_streamed(codes, reinterpret_cast<uint32_t *>(q) + c, stream);
    else
        store_streamed((uint16_t)codes, reinterpret_cast<uint16_t *>(q) + c, stream);
    constexpr int kLanes = 32 / N;
    if (c % kLanes == 0) {
        const int b = c / kLanes, blocks = chunks / kLanes;
        scale[b] = finite ? (uint8_t)e : (uint8_t)255;
        if (b == blocks - 1)
            for (int i = blocks; i % 4 != 0; ++i) scale[i] = 0;
    }
}

}  // namespace emit
}  // namespace moonep
