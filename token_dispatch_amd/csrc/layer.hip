// The whole mixture-of-experts layer for a few tokens in two kernels, for gfx950.
//
//   a[t,k] = silu(G_e x[t]) * (U_e x[t])           e = ids[t,k]
//   out[t] = sum_k w[t,k] D_e a[t,k]
//
// With few tokens the layer is its experts' weights, read once: nothing is planned or moved.
// A distinct expert is a slot. The first kernel's workgroups take 16 rows of G and U of one
// slot, find the slot's tokens in the ids themselves and leave w a of each (token, slot) in
// the workspace; the second's take 16 rows of D of all slots, each of their waves some of
// them, and add the waves' sums up in order. Nothing is atomic.
//
// The weights' rows are the first operand of the matrix units, up to 16 tokens the second:
// with one token 15 columns idle, but the units are far from busy, and lanes without a token
// load nothing. A sum's column holds one token alone, so what an expert's weights or another
// token hold (infinities, NaN) reaches only the tokens that the expert has.
//
// Binary32 values meet weights of fewer bits in pieces of bf16, 8 bits of significand each
// (what is cut off goes to the next piece): 2 for the activations between the kernels where
// rows are bf16, off by 2^-16 at most, and 3 where rows are binary32, off by nothing.
#include "emit.h"
#include "layerops.h"
#include "rows.h"
#include "tiles.h"

namespace moonep {
namespace {

using namespace rows;
using tiles::kOutOfRange;
using tiles::rsrc;
using tiles::v8bf;
using tiles::wave_id;

constexpr int kMaxSlots = 1024;  // experts

// Workspace: the slots' experts (-1: none), the place (k + 1, or 0) of each slot's expert
// among each token's ids, then the pieces of w a, a plane [T*K, F] for each.
constexpr int64_t kMapAt = kMaxSlots * 4;
constexpr int64_t kPlanesAt = kMapAt + (int64_t)kMaxSlots * kFewTokens;

enum Kind { kF32, kBf16, kMxBf16, kMxF32 };

__device__ __forceinline__ v4u load16(__amdgpu_buffer_rsrc_t rs, int at) {
    return __builtin_amdgcn_raw_buffer_load_b128(rs, at, 0, 0);
}

// Weights are read a unit at a time: 16 bytes of each of 16 rows and four places along k, so
// a lane (row l % 16, place l / 16) holds KL values next to each other and a unit is 4 KL
// long. Tokens' values come in the same order along k.
template <int KIND>
struct Unit;

template <>
struct Unit<kF32> {
    static constexpr int KL = 4, kPieces = 1;
    typedef v4u Raw;
    typedef v4f Tokens;
    __device__ static Raw weights(__amdgpu_buffer_rsrc_t rs, __amdgpu_buffer_rsrc_t, int at, int, int) {
        return load16(rs, at);
    }
    __device__ static Tokens rows(__amdgpu_buffer_rsrc_t rs, int at) {
        return __builtin_bit_cast(v4f, load16(rs, at));
    }
    __device__ static Tokens pieces(__amdgpu_buffer_rsrc_t rs, int at, int) { return rows(rs, at); }
    __device__ static v4f mma(const Raw &w, const Tokens &x, v4f c) {
        const v4f a = __builtin_bit_cast(v4f, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], x[j], c, 0, 0, 0);
        return c;
    }
};

template <>
struct Unit<kBf16> {
    static constexpr int KL = 8, kPieces = 2;
    typedef v4u Raw;
    struct Tokens {
        v4u p[2];
        int n;
    };
    __device__ static Raw weights(__amdgpu_buffer_rsrc_t rs, __amdgpu_buffer_rsrc_t, int at, int, int) {
        return load16(rs, at);
    }
    __device__ static Tokens rows(__amdgpu_buffer_rsrc_t rs, int at) { return {{load16(rs, at)}, 1}; }
    __device__ static Tokens pieces(__amdgpu_buffer_rsrc_t rs, int at, int plane) {
        return {{load16(rs, at), load16(rs, at < kOutOfRange ? at + plane : at)}, 2};
    }
    __device__ static v4f mma(const Raw &w, const Tokens &x, v4f c) {
        const v8bf a = __builtin_bit_cast(v8bf, w);
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(v8bf, x.p[0]), c, 0, 0, 0);
        if (x.n > 1)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(v8bf, x.p[1]), c, 0, 0, 0);
        return c;
    }
};

// A lane's 16 bytes are a block of 32 values: four products of 8 along k.
template <int P>
struct Scaled {
    static constexpr int KL = 32, kPieces = P;
    struct Raw {
        v4u q;
        uint32_t scale;  // the byte of this lane's block at the bottom
    };
    struct Tokens {
        v4u p[P][4];
        int n;
    };
    __device__ static Raw weights(__amdgpu_buffer_rsrc_t rs, __amdgpu_buffer_rsrc_t scales, int at,
                                  int scale_at, int shift) {
        return {load16(rs, at),
                (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(scales, scale_at, 0, 0) >> shift & 0xffu};
    }
    __device__ static Tokens pieces(__amdgpu_buffer_rsrc_t rs, int at, int plane) {
        Tokens t;
        t.n = P;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                t.p[p][j] = load16(rs, at < kOutOfRange ? at + p * plane + j * 16 : at);
        return t;
    }
    __device__ static v4f mma(const Raw &w, const Tokens &x, v4f c) {
        const float scale = __uint_as_float(w.scale << 23);  // 255: the conversion gives NaN
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t d = w.q[j];
            v2bf b[4];
            b[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0);
            b[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1);
            b[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2);
            b[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3);
            const v8bf a = {b[0].x, b[0].y, b[1].x, b[1].y, b[2].x, b[2].y, b[3].x, b[3].y};
#pragma unroll
            for (int p = 0; p < P; ++p)
                if (p < x.n)
                    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        a, __builtin_bit_cast(v8bf, x.p[p][j]), c, 0, 0, 0);
        }
        return c;
    }
};

// The high 16 bits of two binary32 values, a's low: their first bf16 pieces.
__device__ __forceinline__ uint32_t high16(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// A NaN whose set bits are all among the low 16 would pass for an infinity in its first piece.
__device__ __forceinline__ float quiet(float v) {
    return v != v ? __uint_as_float(0x7fc00000u) : v;
}

// What the first piece leaves, for the next; nothing where it is infinite or NaN.
__device__ __forceinline__ float rest(float v) {
    const float r = v - __uint_as_float(__float_as_uint(v) & 0xffff0000u);
    return (__float_as_uint(v) & 0x7fffffffu) < emit::kInfBits ? r : 0.0f;
}

template <>
struct Unit<kMxBf16> : Scaled<2> {
    __device__ static Tokens rows(__amdgpu_buffer_rsrc_t rs, int at) {
        Tokens t;
        t.n = 1;
#pragma unroll
        for (int j = 0; j < 4; ++j) t.p[0][j] = load16(rs, at < kOutOfRange ? at + j * 16 : at);
        return t;
    }
};

template <>
struct Unit<kMxF32> : Scaled<3> {
    __device__ static Tokens rows(__amdgpu_buffer_rsrc_t rs, int at) {
        Tokens t;
        t.n = 3;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float v[8];
            Chunk<false>::unpack(load16(rs, at < kOutOfRange ? at + j * 32 : at), v);
            Chunk<false>::unpack(load16(rs, at < kOutOfRange ? at + j * 32 + 16 : at), v + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = quiet(v[i]);
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                t.p[p][j] = v4u{high16(v[0], v[1]), high16(v[2], v[3]), high16(v[4], v[5]), high16(v[6], v[7])};
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = rest(v[i]);
            }
        }
        return t;
    }
};

template <int KIND>
constexpr bool kScaled = KIND == kMxBf16 || KIND == kMxF32;
template <int KIND>
constexpr int kRowBytes = KIND == kBf16 || KIND == kMxBf16 ? 2 : 4;  // of an element of x and out
template <int KIND>
constexpr int kPlaneBytes = KIND == kF32 ? 4 : 2;  // of an element of the workspace's planes

// Bytes of n weights, and of a lane's part of a unit of tokens' values of b bytes each.
template <int KIND>
__device__ __forceinline__ int weight_bytes(int n) {
    return KIND == kBf16 ? n * 2 : KIND == kF32 ? n * 4 : n / 2;
}

// 16 rows of a matrix [n, k] from row `first` on, as a lane reads them.
template <int KIND>
struct Rows16 {
    __amdgpu_buffer_rsrc_t rs, scales;
    int at, scale_at, k, place;

    __device__ void init(const char *w, const uint8_t *scale, int first, int n, int k_) {
        k = k_;
        const int bytes = weight_bytes<KIND>(k), left = min(n - first, 16), l = lane_id();
        rs = rsrc(w + (int64_t)first * bytes, left * bytes);
        at = (l & 15) * bytes + (l >> 4) * 16;
        place = (l >> 4) * Unit<KIND>::KL;
        if constexpr (kScaled<KIND>) {
            const int pitch = emit::scale_pitch(k);
            scales = rsrc(reinterpret_cast<const char *>(scale) + (int64_t)first * pitch, left * pitch);
            scale_at = (l & 15) * pitch;
        } else {
            scales = rs;
            scale_at = 0;
        }
    }

    __device__ bool has(int unit) const { return unit * (4 * Unit<KIND>::KL) + place < k; }

    __device__ typename Unit<KIND>::Raw load(int unit) const {
        const bool in = has(unit);
        return Unit<KIND>::weights(rs, scales, in ? at + unit * 64 : kOutOfRange,
                                   in ? scale_at + unit * 4 : kOutOfRange, (lane_id() >> 4) * 8);
    }
};

struct FewArgs {
    const int32_t *ids;
    const float *topk_w;
    const char *x, *gate, *up, *down;
    const uint8_t *gate_scale, *up_scale, *down_scale;
    void *out;
    char *work;
    int64_t in_block, out_block, in_scale_block, out_scale_block;  // bytes
    int T, E, K, H, F;
    int slots;  // entry s names slot s's expert where slots < E, else slot s is expert s
};

// The place of a unit's first value for this lane in a row of k values of b bytes, or out of range.
__device__ __forceinline__ int value_at(int row_at, int k_at, int k, int b) {
    return row_at >= 0 && k_at < k ? row_at + k_at * b : kOutOfRange;
}

// NT groups of 16 tokens (columns) of this wave's units: gate and up sums.
template <int KIND, int NT, int UN, int NW>
__device__ void gate_up(const FewArgs &a, const Rows16<KIND> &gate, const Rows16<KIND> &up,
                        const int *tokens, int n, v4f (&acc)[NT][2]) {
    typedef Unit<KIND> U;
    const __amdgpu_buffer_rsrc_t xs = rsrc(a.x, a.T * a.H * kRowBytes<KIND>);
    int row[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int col = t * 16 + (lane_id() & 15);
        row[t] = col < n ? tokens[col] * a.H * kRowBytes<KIND> : -1;
        acc[t][0] = acc[t][1] = v4f{0, 0, 0, 0};
    }
    const int units = (a.H + 4 * U::KL - 1) / (4 * U::KL);
    for (int u0 = wave_id() * UN; u0 < units; u0 += NW * UN) {
        typename U::Raw wg[UN], wu[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            wg[i] = gate.load(u0 + i);
            wu[i] = up.load(u0 + i);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t * 16 >= n) break;
            typename U::Tokens x[UN];
#pragma unroll
            for (int i = 0; i < UN; ++i)
                x[i] = U::rows(xs, value_at(row[t], (u0 + i) * 4 * U::KL + gate.place, a.H,
                                            kRowBytes<KIND>));
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                acc[t][0] = U::mma(wg[i], x[i], acc[t][0]);
                acc[t][1] = U::mma(wu[i], x[i], acc[t][1]);
            }
        }
    }
}

// 16 columns of w a for the tokens of a slot.
template <int KIND, int NT, int UN, int NW>
__global__ __launch_bounds__(NW * 64) void k_few_in(FewArgs a) {
    __shared__ int tokens[kFewTokens], entries[kFewTokens];
    __shared__ float weights[kFewTokens];
    __shared__ int count;
    __shared__ v4f sums[NW][NT * 2][64];
    const int slot = blockIdx.y, l = lane_id();
    const bool named = a.slots < a.E;
    const int e = named ? a.ids[slot] : slot;
    if (wave_id() == 0) {
        // lane t: token t's place of the expert and its weight, repeated ids added up
        int place = 0;
        float w = 0;
        if (l < a.T)
            for (int k = 0; k < a.K; ++k)
                if (a.ids[l * a.K + k] == e) {
                    if (place == 0) place = k + 1;
                    w += a.topk_w[l * a.K + k];
                }
        const uint64_t has = __ballot(place > 0);
        const int first = has ? __ffsll((unsigned long long)has) - 1 : 0;
        // a named slot is its expert's first entry's
        const bool mine = e >= 0 && e < a.E && has &&
                          (!named || slot == first * a.K + __builtin_amdgcn_readlane(place, first) - 1);
        if (place > 0) {
            const int i = __popcll(has & ((1ull << l) - 1));
            tokens[i] = l;
            entries[i] = l * a.K + place - 1;
            weights[i] = w;
        }
        if (l == 0) count = mine ? __popcll(has) : 0;
        if (blockIdx.x == 0) {
            if (l == 0) reinterpret_cast<int *>(a.work)[slot] = mine ? e : -1;
            a.work[kMapAt + slot * kFewTokens + l] = (char)(mine ? place : 0);
        }
    }
    __syncthreads();
    const int n = count;
    if (n == 0) return;
    const int f0 = blockIdx.x * 16;
    Rows16<KIND> gate, up;
    gate.init(a.gate + e * a.in_block, a.gate_scale + e * a.in_scale_block, f0, a.F, a.H);
    up.init(a.up + e * a.in_block, a.up_scale + e * a.in_scale_block, f0, a.F, a.H);
    v4f acc[NT][2];
    gate_up<KIND, NT, UN, NW>(a, gate, up, tokens, n, acc);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        sums[wave_id()][t * 2][l] = acc[t][0];
        sums[wave_id()][t * 2 + 1][l] = acc[t][1];
    }
    __syncthreads();
    const int64_t plane = (int64_t)a.T * a.K * a.F;
    for (int t = wave_id(); t < NT; t += NW) {
        v4f g = sums[0][t * 2][l], u = sums[0][t * 2 + 1][l];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
            g += sums[w][t * 2][l];
            u += sums[w][t * 2 + 1][l];
        }
        const int col = t * 16 + (l & 15), f = f0 + (l >> 4) * 4;
        if (col >= n || f >= a.F) continue;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = g[j] / (1.0f + expf(-g[j])) * u[j] * weights[col];
        char *to = a.work + kPlanesAt + ((int64_t)entries[col] * a.F + f) * kPlaneBytes<KIND>;
        if constexpr (KIND == kF32) {
            *reinterpret_cast<v4f *>(to) = v4f{v[0], v[1], v[2], v[3]};
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = quiet(v[j]);
#pragma unroll
            for (int p = 0; p < Unit<KIND>::kPieces; ++p) {
                if (p < Unit<KIND>::kPieces - 1 || p == 2)
                    *reinterpret_cast<v2u *>(to + p * plane * 2) = v2u{high16(v[0], v[1]), high16(v[2], v[3])};
                else  // the last of two is rounded
                    *reinterpret_cast<v2u *>(to + p * plane * 2) =
                        v2u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = rest(v[j]);
            }
        }
    }
}

// 16 columns of out, NT groups of 16 tokens.
template <int KIND, int NT, int UN, int NW>
__global__ __launch_bounds__(NW * 64) void k_few_out(FewArgs a) {
    typedef Unit<KIND> U;
    __shared__ int list[kMaxSlots];  // slots that have an expert
    __shared__ int before[NW + 1];
    __shared__ v4f sums[NW][NT][64];
    const int l = lane_id(), w = wave_id(), n0 = blockIdx.x * 16;
    const int *experts = reinterpret_cast<const int *>(a.work);
    constexpr int kEach = (kMaxSlots + NW * 64 - 1) / (NW * 64);
    // slots in order, kEach next to each other a lane
    int found = 0, mine[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int s = (int)threadIdx.x * kEach + i;
        mine[i] = s < a.slots && experts[s] >= 0;
        found += mine[i];
    }
    int upto = found;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int v = __shfl_up(upto, d);
        if (l >= d) upto += v;
    }
    if (l == 63) before[w + 1] = upto;
    __syncthreads();
    int at = upto - found, n = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        if (i < w) at += before[i + 1];
        n += before[i + 1];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (mine[i]) list[at++] = (int)threadIdx.x * kEach + i;
    __syncthreads();

    v4f acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = v4f{0, 0, 0, 0};
    const int plane = a.T * a.K * a.F * kPlaneBytes<KIND>;
    const __amdgpu_buffer_rsrc_t hs = rsrc(a.work + kPlanesAt, plane * U::kPieces);
    const int units = (a.F + 4 * U::KL - 1) / (4 * U::KL), parts = (units + UN - 1) / UN;
    for (int q = w; q < n * parts; q += NW) {
        const int slot = __builtin_amdgcn_readfirstlane(list[q / parts]), u0 = q % parts * UN;
        const int e = __builtin_amdgcn_readfirstlane(experts[slot]);
        Rows16<KIND> down;
        down.init(a.down + e * a.out_block, a.down_scale + e * a.out_scale_block, n0, a.H, a.F);
        typename U::Raw wd[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) wd[i] = down.load(u0 + i);
        const uint8_t *map = reinterpret_cast<const uint8_t *>(a.work) + kMapAt + slot * kFewTokens;
        int place[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) place[t] = map[t * 16 + (l & 15)];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (__ballot(place[t] > 0) == 0) continue;
            const int entry = (t * 16 + (l & 15)) * a.K + place[t] - 1;
            const int row = place[t] > 0 ? entry * a.F * kPlaneBytes<KIND> : -1;
            typename U::Tokens x[UN];
#pragma unroll
            for (int i = 0; i < UN; ++i)
                x[i] = U::pieces(hs, value_at(row, (u0 + i) * 4 * U::KL + down.place, a.F, kPlaneBytes<KIND>),
                                 plane);
            v4f d = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < UN; ++i) d = U::mma(wd[i], x[i], d);
            // 0 times an infinite weight is NaN: only the expert's own tokens take the sums
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[t][j] += place[t] > 0 ? d[j] : 0.0f;
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) sums[w][t][l] = acc[t];
    __syncthreads();
    for (int t = w; t < NT; t += NW) {
        v4f v = sums[0][t][l];
#pragma unroll
        for (int i = 1; i < NW; ++i) v += sums[i][t][l];
        const int token = t * 16 + (l & 15), col = n0 + (l >> 4) * 4;
        if (token >= a.T || col >= a.H) continue;
        const int64_t to = (int64_t)token * a.H + col;
        const float f[4] = {v[0], v[1], v[2], v[3]};
        store_elems<4, kRowBytes<KIND> == 2, false>(a.out, to, f);
    }
}

template <int KIND, int NT>
hipError_t few_layer(const FewArgs &a, hipStream_t st) {
    constexpr int UN = kScaled<KIND> ? (KIND == kMxF32 ? 1 : 2) : 4;
    constexpr int kIn = 4, kOut = 8;
    hipLaunchKernelGGL((k_few_in<KIND, NT, UN, kIn>), dim3((a.F + 15) / 16, a.slots), dim3(kIn * 64), 0,
                       st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_few_out<KIND, NT, UN, kOut>), dim3((a.H + 15) / 16), dim3(kOut * 64), 0, st, a);
    return hipGetLastError();
}

template <int KIND>
hipError_t few_layer_of(const FewArgs &a, hipStream_t st) {
    if (a.T <= 16) return few_layer<KIND, 1>(a, st);
    if (a.T <= 32) return few_layer<KIND, 2>(a, st);
    return few_layer<KIND, 4>(a, st);
}

}  // namespace

int64_t few_layer_bytes(int32_t T, int32_t E, int32_t K, int32_t F) {
    return kPlanesAt + (int64_t)T * K * F * 6;
}

hipError_t launch_few_layer(const FewLayer &l, hipStream_t st) {
    const int es = l.bf16 ? 2 : 4;
    const bool scaled = l.gate_scale != nullptr;
    FewArgs a;
    a.ids = l.ids;
    a.topk_w = l.topk_w;
    a.x = static_cast<const char *>(l.x);
    a.gate = static_cast<const char *>(l.gate);
    a.up = static_cast<const char *>(l.up);
    a.down = static_cast<const char *>(l.down);
    a.gate_scale = l.gate_scale;
    a.up_scale = l.up_scale;
    a.down_scale = l.down_scale;
    a.out = l.out;
    a.work = static_cast<char *>(l.work);
    a.in_block = l.in_block * (scaled ? 1 : es);
    a.out_block = l.out_block * (scaled ? 1 : es);
    a.in_scale_block = l.in_scale_block;
    a.out_scale_block = l.out_scale_block;
    a.T = l.T;
    a.E = l.E;
    a.K = l.K;
    a.H = l.H;
    a.F = l.F;
    a.slots = l.T * l.K < l.E ? l.T * l.K : l.E;
    if (scaled) return l.bf16 ? few_layer_of<kMxBf16>(a, st) : few_layer_of<kMxF32>(a, st);
    return l.bf16 ? few_layer_of<kBf16>(a, st) : few_layer_of<kF32>(a, st);
}

}  // namespace moonep
