// The global norm of many gradient tensors and their clipping, for gfx950.
//
//   sumsq = sum over all tensors of g^2, binary64
//   norm  = sqrt(sumsq);  c = max_norm / norm where norm > max_norm, else 1
//   out   = g * c
//
// Bound by HBM: the gradients are read twice and written once (1.6 GB of binary32: the
// norm 0.27 ms, 6.0 TB/s, the clipping 0.57 ms, 5.6 TB/s). The tensors of one
// launch travel in its arguments (no table in device memory, so a captured launch
// keeps its own). They are cut into chunks; workgroup w of the norm's launch adds
// chunks w, w + grid, ... in that order into its own slot, and one workgroup adds
// the slots in order, so equal inputs give equal bits and nothing is atomic.
#include "experts.h"
#include "rows.h"

namespace moonep {
namespace {

using namespace rows;

constexpr int kThreads = 256;
constexpr int kList = 128;  // tensors one launch's arguments hold
constexpr int kSlots = MOONEP_NORM_DOUBLES - 1;

// Chunks of 2^shift elements: 64 KB of binary32 for large sets (a few hundred cycles of
// look-up for each), down to 2^10 elements for small ones, so that those too spread over
// the device.
constexpr int kMaxShift = 14, kMinShift = 10;

struct List {
    const void *in[kList];
    void *out[kList];
    int32_t end[kList];  // chunks of tensors 0 .. i together
    int64_t numel[kList];
    uint32_t bf16[kList / 32];
    int32_t n, shift;
    int32_t stream;  // outputs go past the caches
};

struct Chunk {
    const char *in;
    char *out;
    int len;
    bool bf16;
};

__device__ __forceinline__ Chunk chunk_at(const List &l, int c) {
    int lo = 0, hi = l.n - 1;  // the first tensor whose chunks end past c
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (l.end[mid] > c) hi = mid;
        else lo = mid + 1;
    }
    const int64_t at = (int64_t)(c - (lo > 0 ? l.end[lo - 1] : 0)) << l.shift;
    const bool bf16 = l.bf16[lo / 32] >> (lo % 32) & 1;
    const int64_t left = l.numel[lo] - at;
    const int es = bf16 ? 2 : 4;
    return {static_cast<const char *>(l.in[lo]) + at * es, static_cast<char *>(l.out[lo]) + at * es,
            (int)(left < 1 << l.shift ? left : 1 << l.shift), bf16};
}

// 16 bytes at an element's alignment, as a gradient that is a view of a larger buffer has.
template <bool BF16>
struct Elems;
template <>
struct Elems<true> {
    static constexpr int N = 8;
    typedef uint16_t T;
    typedef uint32_t __attribute__((ext_vector_type(4), aligned(2))) V;
    __device__ static float one(T v) { return __uint_as_float((uint32_t)v << 16); }
    __device__ static T round(float v) { return (T)(pack_bf16x2(v, 0.0f) & 0xffffu); }
};
template <>
struct Elems<false> {
    static constexpr int N = 4;
    typedef float T;
    typedef uint32_t __attribute__((ext_vector_type(4), aligned(4))) V;
    __device__ static float one(T v) { return v; }
    __device__ static T round(float v) { return v; }
};

// Sum of squares of one thread's part of `len` elements. Four sums, added in their order.
template <bool BF16>
__device__ __forceinline__ double squares(const char *in, int len) {
    typedef Elems<BF16> E;
    typedef typename E::V V;
    constexpr int N = E::N, kUnroll = 4;
    double s[4] = {0, 0, 0, 0};
    const int vecs = len / N;
    const V *p = reinterpret_cast<const V *>(in);
    auto add = [&](const V &q) {
        float x[N];
        rows::Chunk<BF16>::unpack(v4u{q.x, q.y, q.z, q.w}, x);
#pragma unroll
        for (int j = 0; j < N; ++j) s[j % 4] = __builtin_fma((double)x[j], (double)x[j], s[j % 4]);
    };
    int i = threadIdx.x;
    for (; i + (kUnroll - 1) * kThreads < vecs; i += kUnroll * kThreads) {
        V v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u] = p[i + u * kThreads];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) add(v[u]);
    }
    for (; i < vecs; i += kThreads) add(p[i]);
    const int at = vecs * N + (int)threadIdx.x;
    if (at < len) {
        const double v = E::one(reinterpret_cast<const typename E::T *>(in)[at]);
        s[0] = __builtin_fma(v, v, s[0]);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// A factor m * 2^e. With e = 0, m is the factor in binary32; a factor below the normal binary32
// numbers is split, so that it keeps all of m's digits and products that are normal numbers again
// (of gradients up to 3e38) have two roundings like any others. One more instruction for each
// element, in a kernel that HBM bounds.
struct Factor {
    float m;
    int e;
    __device__ float times(float x) const { return ldexpf(x * m, e); }
};

// out = in * f: element by element up to the first 16-byte boundary of out and behind the
// last, 16 bytes at a time between.
template <bool BF16>
__device__ __forceinline__ void scaled(const char *in, char *out, int len, Factor f, bool stream) {
    typedef Elems<BF16> E;
    typedef typename E::V V;
    typedef typename E::T T;
    constexpr int N = E::N, kUnroll = 4;
    const T *p = reinterpret_cast<const T *>(in);
    T *o = reinterpret_cast<T *>(out);
    const int head = min(len, (int)((0 - reinterpret_cast<uintptr_t>(out)) % 16 / sizeof(T)));
    const int vecs = (len - head) / N, tail = head + vecs * N;
    const int t = threadIdx.x;
    if (t < head) o[t] = E::round(f.times(E::one(p[t])));
    if (tail + t < len) o[tail + t] = E::round(f.times(E::one(p[tail + t])));
    const V *pv = reinterpret_cast<const V *>(p + head);
    auto put = [&](int i, const V &q) {
        float x[N];
        rows::Chunk<BF16>::unpack(v4u{q.x, q.y, q.z, q.w}, x);
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = f.times(x[j]);
        v4u out;
        if constexpr (BF16)
            out = v4u{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7])};
        else
            out = v4u{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3])};
        store_streamed(out, reinterpret_cast<v4u *>(o + head) + i, stream);
    };
    int i = t;
    for (; i + (kUnroll - 1) * kThreads < vecs; i += kUnroll * kThreads) {
        V v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u] = __builtin_nontemporal_load(pv + i + u * kThreads);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) put(i + u * kThreads, v[u]);
    }
    for (; i < vecs; i += kThreads) put(i, pv[i]);
}

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double s[kThreads / 64];
    for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
    __syncthreads();
    if (lane_id() == 0) s[threadIdx.x / 64] = v;
    __syncthreads();
    double t = 0;
    for (int i = 0; i < kThreads / 64; ++i) t += s[i];
    return t;
}

__global__ __launch_bounds__(kThreads) void k_sumsq(List l, double *slots, int filled) {
    double sum = 0;
    const int chunks = l.end[l.n - 1];
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Chunk ch = chunk_at(l, c);
        sum += ch.bf16 ? squares<true>(ch.in, ch.len) : squares<false>(ch.in, ch.len);
    }
    sum = block_sum(sum);
    // slots below `filled` hold sums of the call's earlier launches
    if (threadIdx.x == 0) slots[blockIdx.x] = (int)blockIdx.x < filled ? slots[blockIdx.x] + sum : sum;
}

__global__ __launch_bounds__(kThreads) void k_join(double *acc, int filled) {
    double sum = 0;
    for (int i = threadIdx.x; i < filled; i += kThreads) sum += acc[1 + i];
    sum = block_sum(sum);
    if (threadIdx.x == 0) acc[0] = sum;
}

// The norm is compared in binary64, in which the squares of binary32 numbers do not overflow. A
// finite norm past binary32's range is reported as the largest finite number, so that an infinite
// or NaN report always means that the gradients were left as they are.
__device__ __forceinline__ Factor clip_factor(double sumsq, double max_norm, float *norm) {
    const double n = sqrt(sumsq);
    const bool finite = n < __longlong_as_double(0x7ff0000000000000ll);  // false for a NaN
    *norm = finite ? fminf((float)n, 3.402823466e38f) : (float)n;
    if (!(finite && n > max_norm)) return {1.0f, 0};
    const double c = max_norm / n;
    if (c >= 0x1p-126) return {(float)c, 0};
    int e;
    const double m = frexp(c, &e);
    return {(float)m, e};
}

__global__ __launch_bounds__(kThreads) void k_clip(List l, const double *acc, double max_norm,
                                                   float *norm) {
    float n;
    const Factor f = clip_factor(acc[0], max_norm, &n);
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
    const int chunks = l.n > 0 ? l.end[l.n - 1] : 0;
    // from the last chunk to the first: the norm's pass left the last ones in the cache
    for (int c = chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
        const Chunk ch = chunk_at(l, c);
        if (f.m == 1.0f && f.e == 0 && ch.in == ch.out) continue;
        if (ch.bf16) scaled<true>(ch.in, ch.out, ch.len, f, l.stream);
        else scaled<false>(ch.in, ch.out, ch.len, f, l.stream);
    }
}

// What a call's launches share: the elements of one chunk, as a shift (about two chunks for
// each slot), and whether outputs go past the caches.
void begin(List &l, int32_t n, const int64_t *numel, const int32_t *dtypes) {
    int64_t total = 0, bytes = 0;
    for (int32_t i = 0; i < n; ++i) {
        total += numel[i];
        bytes += numel[i] * (dtypes[i] == MOONEP_BF16 ? 2 : 4);
    }
    l.shift = kMinShift;
    while (l.shift < kMaxShift && (total >> l.shift) > 2 * kSlots) ++l.shift;
    l.stream = bytes >= kStreamBytes;
}

// Fills one launch's list with tensors from `at` on; returns where it stopped.
int32_t fill(List &l, int32_t at, int32_t n, const void *const *in, void *const *out,
             const int64_t *numel, const int32_t *dtypes) {
    l.n = 0;
    for (uint32_t &w : l.bf16) w = 0;
    int64_t chunks = 0;
    for (; at < n && l.n < kList; ++at) {
        if (numel[at] == 0) continue;
        const int64_t more = (numel[at] + (1 << l.shift) - 1) >> l.shift;
        if (chunks + more >= ((int64_t)1 << 31) - (1 << 16)) break;
        chunks += more;
        l.in[l.n] = in[at];
        l.out[l.n] = out != nullptr ? out[at] : nullptr;
        l.end[l.n] = (int32_t)chunks;
        l.numel[l.n] = numel[at];
        if (dtypes[at] == MOONEP_BF16) l.bf16[l.n / 32] |= 1u << (l.n % 32);
        ++l.n;
    }
    return at;
}

}  // namespace

hipError_t launch_grad_sumsq(int32_t n, const void *const *grads, const int64_t *numel,
                             const int32_t *dtypes, double *acc, hipStream_t st) {
    List l;
    begin(l, n, numel, dtypes);
    int filled = 0;
    for (int32_t at = 0; at < n;) {
        at = fill(l, at, n, grads, nullptr, numel, dtypes);
        if (l.n == 0) break;
        const int chunks = l.end[l.n - 1], grid = chunks < kSlots ? chunks : kSlots;
        hipLaunchKernelGGL(k_sumsq, dim3(grid), dim3(kThreads), 0, st, l, acc + 1, filled);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (grid > filled) filled = grid;
    }
    hipLaunchKernelGGL(k_join, dim3(1), dim3(kThreads), 0, st, acc, filled);
    return hipGetLastError();
}

hipError_t launch_grad_clip(int32_t n, const void *const *grads, void *const *outs,
                            const int64_t *numel, const int32_t *dtypes, const double *acc,
                            double max_norm, float *norm, hipStream_t st) {
    List l;
    l.n = 0;
    begin(l, n, numel, dtypes);
    for (int32_t at = 0; at < n || norm != nullptr;) {
        at = fill(l, at, n, grads, outs, numel, dtypes);
        if (l.n == 0 && norm == nullptr) break;
        const int chunks = l.n > 0 ? l.end[l.n - 1] : 1, grid = chunks < kSlots ? chunks : kSlots;
        hipLaunchKernelGGL(k_clip, dim3(grid), dim3(kThreads), 0, st, l, acc, max_norm, norm);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        norm = nullptr;  // the first launch writes it
    }
    return hipSuccess;
}

}  // namespace moonep
