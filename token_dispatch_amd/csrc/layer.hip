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
// Binary32 values, the activations between the kernels and binary32 rows, meet weights of fewer
// bits in three pieces of bf16, 8 bits of significand each (what is cut off goes to the next
// piece, Pieces): all 24 bits from magnitudes of 2^-100 on, below which a piece may pass under
// bf16's normal numbers. Two pieces, the second rounded, changed one bf16 result in 200 against
// binary32's.
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

enum Kind { kF32, kBf16, kMxBf16, kMxF32 };  // weights (and rows, where they differ)

__device__ __forceinline__ v4u load16(__amdgpu_buffer_rsrc_t rs, int at) {
    return __builtin_amdgcn_raw_buffer_load_b128(rs, at, 0, 0);
}

// The high 16 bits of two binary32 values, a's low: their bf16 pieces, where the low 16 are zeros.
__device__ __forceinline__ uint32_t high16(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// The three pieces of a value. None is zero, all have its sign and whole numbers of its last
// bit (half of that for a power of two), so that they add up to it in binary32 whatever their
// order, and an infinite weight gives an infinity of the right sign with each of them (zero
// times it would be NaN). A piece is what is left, less enough for those behind it, cut off: two
// last bits for the first, one for the second. A zero, an infinity or NaN is all of its pieces.
struct Pieces {
    float left, below;  // what is left, and the same of the value's neighbour towards zero
    bool number;

    __device__ explicit Pieces(float v) {
        const uint32_t bits = __float_as_uint(v);
        number = (bits & 0x7fffffffu) - 2u < emit::kInfBits - 2u;
        // a NaN whose set bits are all among the low 16 would pass for an infinity
        left = v != v ? __uint_as_float(0x7fc00000u) : v;
        below = __uint_as_float(bits - 1u);
    }

    template <int P>
    __device__ float piece() {
        if (P == 2 || !number) return left;
        const uint32_t bits = P == 0 ? __float_as_uint(left) - 2u : __float_as_uint(below);
        const float p = __uint_as_float(bits & 0xffff0000u);
        left -= p;
        below -= p;
        return p;
    }
};

// Piece P of some values, two to a word.
template <int P, int N>
__device__ __forceinline__ void put_pieces(Pieces (&v)[N], uint32_t (&out)[N / 2]) {
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = v[i].template piece<P>();
#pragma unroll
    for (int i = 0; i < N / 2; ++i) out[i] = high16(f[2 * i], f[2 * i + 1]);
}

// Weights are read a unit at a time: 16 bytes of each of 16 rows and four places along k, so
// a lane (row l % 16, place l / 16) holds KL values next to each other and a unit is 4 KL
// long. The tokens' values, the other operand, come in the same order along k: fragments of
// 16 bytes a lane (column l % 16, place l / 16), J of them for a unit, in P pieces.
template <int KIND>
struct Unit;

template <>
struct Unit<kF32> {
    static constexpr int KL = 4, J = 1, kIn = 1, kOut = 1, kRow = 4, kPlane = 4;
    template <int P>
    __device__ static v4f mma(const v4u &w, uint32_t, const v4u (&x)[P][J], v4f c) {
        const v4f a = __builtin_bit_cast(v4f, w), b = __builtin_bit_cast(v4f, x[0][0]);
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
        return c;
    }
};

template <>
struct Unit<kBf16> {
    static constexpr int KL = 8, J = 1, kIn = 1, kOut = 3, kRow = 2, kPlane = 2;
    template <int P>
    __device__ static v4f mma(const v4u &w, uint32_t, const v4u (&x)[P][J], v4f c) {
#pragma unroll
        for (int p = 0; p < P; ++p)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, w),
                                                        __builtin_bit_cast(v8bf, x[p][0]), c, 0, 0, 0);
        return c;
    }
};

// A lane's 16 bytes are a block of 32 values, whose scale is a byte: four products of 8 along k.
struct Scaled {
    static constexpr int KL = 32, J = 4;
    template <int P>
    __device__ static v4f mma(const v4u &w, uint32_t byte, const v4u (&x)[P][J], v4f c) {
        const float scale = __uint_as_float(byte << 23);  // 255: the conversion gives NaN
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t d = w[j];
            const v2bf b0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0);
            const v2bf b1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1);
            const v2bf b2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2);
            const v2bf b3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3);
            const v8bf a = {b0.x, b0.y, b1.x, b1.y, b2.x, b2.y, b3.x, b3.y};
#pragma unroll
            for (int p = 0; p < P; ++p)
                c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(v8bf, x[p][j]), c, 0,
                                                            0, 0);
        }
        return c;
    }
};
template <>
struct Unit<kMxBf16> : Scaled {
    static constexpr int kIn = 1, kOut = 3, kRow = 2, kPlane = 2;
};
template <>
struct Unit<kMxF32> : Scaled {
    static constexpr int kIn = 3, kOut = 3, kRow = 4, kPlane = 2;
};

template <int KIND>
constexpr bool kScaled = KIND == kMxBf16 || KIND == kMxF32;

// Bytes of a row of n weights.
template <int KIND>
__device__ __forceinline__ int weight_bytes(int n) {
    return KIND == kBf16 ? n * 2 : KIND == kF32 ? n * 4 : n / 2;
}

// 16 rows of a matrix [n, k] from row `first` on (none from n on), as a lane reads them.
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
        }
    }

    __device__ bool has(int unit) const { return unit * (4 * Unit<KIND>::KL) + place < k; }

    __device__ v4u codes(int unit) const { return load16(rs, has(unit) ? at + unit * 64 : kOutOfRange); }

    // The word that holds the scales of a unit, nothing where this lane's block is behind the
    // row, whose byte may hold anything; or of four units of rows of whole fours.
    __device__ uint32_t word(int unit) const {
        return __builtin_amdgcn_raw_buffer_load_b32(scales, has(unit) ? scale_at + unit * 4 : kOutOfRange, 0, 0);
    }
    __device__ v4u words(int unit) const {
        return load16(scales, has(unit) ? scale_at + unit * 4 : kOutOfRange);
    }
};

// 16 TR rows of a matrix, and UN units of them from unit u0 on. WIDE: rows are whole groups of
// four units, whose scales come in one load (with one load a unit the scales took a third of the
// first kernel's time: 117 us, 81 without them, at 8 tokens of 896 experts of 7168 x 512).
template <int KIND, int TR>
struct Rows {
    Rows16<KIND> part[TR];

    __device__ void init(const char *w, const uint8_t *scale, int first, int n, int k) {
#pragma unroll
        for (int r = 0; r < TR; ++r) part[r].init(w, scale, min(first + r * 16, n), n, k);
    }
};

template <int KIND, int TR, int UN, bool WIDE>
struct Units {
    static_assert(!WIDE || UN % 4 == 0, "groups of four");
    v4u q[TR][UN];
    uint32_t s[TR][kScaled<KIND> ? UN : 1];

    __device__ void load(const Rows<KIND, TR> &rows, int u0) {
#pragma unroll
        for (int r = 0; r < TR; ++r) {
#pragma unroll
            for (int i = 0; i < UN; ++i) q[r][i] = rows.part[r].codes(u0 + i);
            if constexpr (kScaled<KIND>) {
#pragma unroll
                for (int i = 0; i < UN; i += WIDE ? 4 : 1) {
                    if constexpr (WIDE) {
                        const v4u t = rows.part[r].words(u0 + i);
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[r][i + j] = t[j];
                    } else {
                        s[r][i] = rows.part[r].word(u0 + i);
                    }
                }
            }
        }
    }

    template <int P>
    __device__ v4f mma(int r, int i, const v4u (&x)[P][Unit<KIND>::J], v4f c) const {
        uint32_t byte = 0;
        if constexpr (kScaled<KIND>) byte = s[r][i] >> (lane_id() >> 4) * 8 & 0xffu;
        return Unit<KIND>::mma(q[r][i], byte, x, c);
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

// A fragment of the tokens' values: 16 bytes of each of P pieces from value k of a row at
// byte `row` (out of range from value n on), read from the layer's input or from the planes.
template <int KIND>
__device__ __forceinline__ void input_fragment(__amdgpu_buffer_rsrc_t rs, int row, int k, int n,
                                               v4u (&x)[Unit<KIND>::kIn]) {
    const int at = row >= 0 && k < n ? row + k * Unit<KIND>::kRow : kOutOfRange;
    if constexpr (KIND == kMxF32) {
        float v[8];
        Chunk<false>::unpack(load16(rs, at), v);
        Chunk<false>::unpack(load16(rs, at < kOutOfRange ? at + 16 : at), v + 4);
        Pieces of[8] = {Pieces(v[0]), Pieces(v[1]), Pieces(v[2]), Pieces(v[3]),
                        Pieces(v[4]), Pieces(v[5]), Pieces(v[6]), Pieces(v[7])};
        tiles::each<3>([&](auto p) {
            uint32_t w[4];
            put_pieces<decltype(p)::value>(of, w);
            x[decltype(p)::value] = v4u{w[0], w[1], w[2], w[3]};
        });
    } else {
        x[0] = load16(rs, at);
    }
}

template <int KIND>
__device__ __forceinline__ void plane_fragment(__amdgpu_buffer_rsrc_t rs, int row, int k, int n,
                                               int plane, v4u (&x)[Unit<KIND>::kOut]) {
    const int at = row >= 0 && k < n ? row + k * Unit<KIND>::kPlane : kOutOfRange;
#pragma unroll
    for (int p = 0; p < Unit<KIND>::kOut; ++p)  // out of range whatever the plane is
        x[p] = __builtin_amdgcn_raw_buffer_load_b128(rs, at, p * plane, 0);
}

// Lane I of each 16 in lanes 4 C .. 4 C + 3 of them (C < 0: in all 16), `to` in the others.
template <int I, int C>
__device__ __forceinline__ v4u spread(const v4u &v, const v4u &to) {
    v4u out;
#pragma unroll
    for (int j = 0; j < 4; ++j)  // row_newbcast
        out[j] = (uint32_t)__builtin_amdgcn_update_dpp((int)to[j], (int)v[j], 0x150 + I, 0xf,
                                                       C < 0 ? 0xf : 1 << C, true);
    return out;
}

// One token's fragments of UN units: lane i of each 16 holds fragment i % J of unit i / J, so
// they come in P loads where a load for each would bring a column of 16 only. They are spread
// to the other lanes when their unit is multiplied. (A load takes its time whatever its lanes
// get: with 8 loads for a unit the tokens' values took 19 us of the first kernel's 117, at 8 tokens
// of 896 experts of 7168 x 512 in 4 bits.)
template <int KIND, int P, int UN>
struct Token {
    static constexpr int J = Unit<KIND>::J;
    static_assert(UN * J <= 16, "fragments lie side by side in 16 lanes");
    v4u x[P];

    __device__ static int k_at(int u0) {
        const int i = lane_id() & 15, g = lane_id() >> 4;
        return (u0 + i / J) * (4 * Unit<KIND>::KL) + g * Unit<KIND>::KL + i % J * 8;
    }

    // Unit I's fragments into the columns that token C has, into all where C < 0.
    template <int I, int C>
    __device__ void of_unit(v4u (&f)[P][J]) const {
#pragma unroll
        for (int p = 0; p < P; ++p)
            tiles::each<J>([&](auto at) {
                constexpr int j = decltype(at)::value;
                f[p][j] = spread<I * J + j, C>(x[p], C < 0 ? x[p] : f[p][j]);
            });
    }
};

// Tokens that are loaded one by one. Token c has the columns 4 c .. 4 c + 3, of which the first
// counts: one lane move writes a bank of 4 lanes and leaves the others.
constexpr int kFewColumns = 4;

// Nothing moves across: loads before this are in flight together.
__device__ __forceinline__ void issue() { __builtin_amdgcn_sched_barrier(0); }

// NT groups of 16 tokens (columns; 0: kFewColumns tokens at most) times this wave's units of
// gate and up, UN at a time, NW waves in turn. `g` and `u` hold the first of them. The next
// weights are on their way while the matrix units work on those before.
template <int KIND, int NT, int TR, int UN, int NW, bool WIDE>
__device__ __forceinline__ void gate_up(const FewArgs &a, const Rows<KIND, TR> &gate,
                                        const Rows<KIND, TR> &up, const int *tokens, int n,
                                        Units<KIND, TR, UN, WIDE> g, Units<KIND, TR, UN, WIDE> u,
                                        v4f (&acc)[NT > 0 ? NT : 1][TR][2]) {
    typedef Unit<KIND> U;
    constexpr int P = U::kIn;
    const __amdgpu_buffer_rsrc_t xs = rsrc(a.x, a.T * a.H * U::kRow);
    constexpr int kRows = NT > 0 ? NT : kFewColumns;
    int row[kRows];
#pragma unroll
    for (int t = 0; t < kRows; ++t) {
        const int col = NT > 0 ? t * 16 + (lane_id() & 15) : t;
        row[t] = col < n ? tokens[col] * a.H * U::kRow : -1;
    }
#pragma unroll
    for (int t = 0; t < (NT > 0 ? NT : 1); ++t)
#pragma unroll
        for (int r = 0; r < TR; ++r) acc[t][r][0] = acc[t][r][1] = v4f{0, 0, 0, 0};
    const int units = (a.H + 4 * U::KL - 1) / (4 * U::KL);
    for (int u0 = wave_id() * UN; u0 < units; u0 += NW * UN) {
        Units<KIND, TR, UN, WIDE> next_g, next_u;
        auto next = [&] {
            next_g.load(gate, u0 + NW * UN);
            next_u.load(up, u0 + NW * UN);
            issue();
        };
        auto products = [&](int i, const v4u (&x)[P][U::J], v4f (&c)[TR][2]) {
#pragma unroll
            for (int r = 0; r < TR; ++r) {
                c[r][0] = g.mma(r, i, x, c[r][0]);
                c[r][1] = u.mma(r, i, x, c[r][1]);
            }
        };
        if constexpr (NT == 0) {
            Token<KIND, P, UN> x[kFewColumns];
#pragma unroll
            for (int c = 0; c < kFewColumns; ++c)
                if (c < n) input_fragment<KIND>(xs, row[c], Token<KIND, P, UN>::k_at(u0), a.H, x[c].x);
            next();
            tiles::each<UN>([&](auto at) {
                constexpr int i = decltype(at)::value;
                v4u f[P][U::J];
                x[0].template of_unit<i, -1>(f);
                tiles::each<kFewColumns - 1>([&](auto c) {
                    constexpr int C = decltype(c)::value + 1;
                    if (C < n) x[C].template of_unit<i, C>(f);
                });
                products(i, f, acc[0]);
            });
        } else {
            // units at a time whose fragments, of all groups, are few registers
            constexpr int kAll = NT * P * U::J, kAtOnce = kAll <= 2 && UN % 4 == 0 ? 4 : kAll <= 4 && UN % 2 == 0 ? 2 : 1;
            tiles::each<UN / kAtOnce>([&](auto at) {
                constexpr int i0 = decltype(at)::value * kAtOnce;
                v4u x[kAtOnce][NT][P][U::J];
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int j = 0; j < U::J; ++j) {
                            v4u f[P];
                            input_fragment<KIND>(xs, row[t], (u0 + i0 + i) * 4 * U::KL + gate.part[0].place + j * 8,
                                                 a.H, f);
#pragma unroll
                            for (int p = 0; p < P; ++p) x[i][t][p][j] = f[p];
                        }
                if constexpr (i0 == 0) next();
                else issue();
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
                    for (int t = 0; t < NT; ++t) products(i0 + i, x[i][t], acc[t]);
            });
        }
        g = next_g;
        u = next_u;
    }
}

// 16 TR columns of w a for the tokens of a slot. Bound by HBM where the weights are many: 24 tokens
// of 896 experts of 7168 x 512 in bf16 (some 210 of them have one, 3.1 GB) take 512 us, 6.1 TB/s by the
// counters; by the chain of its loads (ids, weights, sums) where they are few: one token of 8
// experts of 2048 x 1024, 67 MB, 16 us. Weights of 4 bits, 5.0 TB/s (79 us, 8 tokens), leave
// short rows and more work a byte. 16 rows a workgroup: as many workgroups as can be.
template <int KIND, int NT, int TR, int UN, int NW, bool WIDE>
__global__ __launch_bounds__(NW * 64) void k_few_in(FewArgs a) {
    __shared__ int tokens[kFewTokens], entries[kFewTokens];
    __shared__ float weights[kFewTokens];
    __shared__ int count;
    __shared__ v4f sums[NW][NT * TR * 2][64];
    const int slot = blockIdx.y, l = lane_id(), f0 = blockIdx.x * (16 * TR);
    const bool named = a.slots < a.E;
    const int e = __builtin_amdgcn_readfirstlane(named ? a.ids[slot] : slot);
    if (e < 0 || e >= a.E) {  // an id outside the experts
        if (blockIdx.x == 0 && threadIdx.x == 0) reinterpret_cast<int *>(a.work)[slot] = -1;
        return;
    }
    Rows<KIND, TR> gate, up;
    gate.init(a.gate + e * a.in_block, a.gate_scale + e * a.in_scale_block, f0, a.F, a.H);
    up.init(a.up + e * a.in_block, a.up_scale + e * a.in_scale_block, f0, a.F, a.H);
    Units<KIND, TR, UN, WIDE> first_g, first_u;
    auto begin = [&] {
        first_g.load(gate, wave_id() * UN);
        first_u.load(up, wave_id() * UN);
        issue();
    };
    // a named slot most likely has its expert: its weights need not wait for the ids
    if (named) begin();
    if (wave_id() == 0) {
        // lane t: which of token t's entries name the expert, and their weights together
        uint64_t which = 0;
        if (l < a.T) {
            const int *ids = a.ids + l * a.K;
            int k = 0;
            for (; k + 8 <= a.K; k += 8) {
                int id[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) id[i] = ids[k + i];
#pragma unroll
                for (int i = 0; i < 8; ++i) which |= (uint64_t)(id[i] == e) << (k + i);
            }
            for (; k < a.K; ++k) which |= (uint64_t)(ids[k] == e) << k;
        }
        const int place = __ffsll((unsigned long long)which);
        float w = 0;
        for (uint64_t m = which; m; m &= m - 1)
            w += a.topk_w[l * a.K + __ffsll((unsigned long long)m) - 1];
        const uint64_t has = __ballot(place > 0);
        const int owner = has ? __ffsll((unsigned long long)has) - 1 : 0;
        // a named slot is its expert's first entry's
        const bool mine = has && (!named || slot == owner * a.K + __builtin_amdgcn_readlane(place, owner) - 1);
        if (place > 0) {
            const int i = __popcll(has & ((1ull << l) - 1));
            tokens[i] = l;
            entries[i] = l * a.K + place - 1;
            weights[i] = w;
        }
        if (l == 0) count = mine ? __popcll(has) : 0;
        if (blockIdx.x == 0) {
            if (l == 0) reinterpret_cast<int *>(a.work)[slot] = mine ? e : -1;
            a.work[kMapAt + slot * kFewTokens + l] = (char)place;
        }
    }
    __syncthreads();
    const int n = __builtin_amdgcn_readfirstlane(count);
    if (n == 0) return;
    if (!named) begin();
    auto finish = [&](auto &acc, int apart) {  // of a token's column from the next one's
        constexpr int M = sizeof(acc) / sizeof(acc[0]) * TR;  // tiles of 16 rows and 16 tokens
#pragma unroll
        for (int t = 0; t < M; ++t) {
            sums[wave_id()][t * 2][l] = acc[t / TR][t % TR][0];
            sums[wave_id()][t * 2 + 1][l] = acc[t / TR][t % TR][1];
        }
        __syncthreads();
        const int64_t plane = (int64_t)a.T * a.K * a.F;
        for (int t = wave_id(); t < M; t += NW) {
            v4f g = sums[0][t * 2][l], u = sums[0][t * 2 + 1][l];
#pragma unroll
            for (int w = 1; w < NW; ++w) {
                g += sums[w][t * 2][l];
                u += sums[w][t * 2 + 1][l];
            }
            const int at = t / TR * 16 + (l & 15), col = at / apart, f = f0 + t % TR * 16 + (l >> 4) * 4;
            if (at % apart != 0 || col >= n || f >= a.F) continue;
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = g[j] * emit::sigmoid(g[j]) * u[j] * weights[col];
            char *to = a.work + kPlanesAt + ((int64_t)entries[col] * a.F + f) * Unit<KIND>::kPlane;
            if constexpr (KIND == kF32) {
                *reinterpret_cast<v4f *>(to) = v4f{v[0], v[1], v[2], v[3]};
            } else {
                Pieces of[4] = {Pieces(v[0]), Pieces(v[1]), Pieces(v[2]), Pieces(v[3])};
                tiles::each<Unit<KIND>::kOut>([&](auto p) {
                    uint32_t w[2];
                    put_pieces<decltype(p)::value>(of, w);
                    *reinterpret_cast<v2u *>(to + decltype(p)::value * plane * 2) = v2u{w[0], w[1]};
                });
            }
        }
    };
    if (n <= kFewColumns) {
        v4f acc[1][TR][2];
        gate_up<KIND, 0, TR, UN, NW, WIDE>(a, gate, up, tokens, n, first_g, first_u, acc);
        finish(acc, 16 / kFewColumns);
    } else if (n <= 16) {
        v4f acc[1][TR][2];
        gate_up<KIND, 1, TR, UN, NW, WIDE>(a, gate, up, tokens, n, first_g, first_u, acc);
        finish(acc, 1);
    } else if constexpr (NT > 1) {
        v4f acc[NT][TR][2];
        gate_up<KIND, NT, TR, UN, NW, WIDE>(a, gate, up, tokens, n, first_g, first_u, acc);
        finish(acc, 1);
    }
}

// 16 TR columns of out, NT groups of 16 tokens. The sum over slots is what keeps a workgroup to its
// rows of all of them: a split over slots would want a third kernel to join them, or atomics.
// 1.46 GB of D in bf16 248 us, 5.9 TB/s by the counters; 186 MB in 4 bits 59 us, 3.2 TB/s, where rows of
// 512 values are 256 bytes; one token's 8 slots, 34 MB, 13 us, most of it the list of slots, the
// first loads and the waves' sums.
template <int KIND, int NT, int TR, int UN, int NW, bool WIDE>
__global__ __launch_bounds__(NW * 64) void k_few_out(FewArgs a) {
    typedef Unit<KIND> U;
    constexpr int P = U::kOut;
    __shared__ int list[kMaxSlots];  // slots that have an expert, and that
    __shared__ int before[NW];
    __shared__ v4f sums[NW][NT * TR][64];
    const int l = lane_id(), w = wave_id(), n0 = blockIdx.x * (16 * TR);
    const int *experts = reinterpret_cast<const int *>(a.work);
    constexpr int kEach = (kMaxSlots + NW * 64 - 1) / (NW * 64);
    // slots in order, kEach next to each other a lane
    int found = 0, mine[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int s = (int)threadIdx.x * kEach + i;
        mine[i] = s < a.slots ? experts[s] : -1;
        found += mine[i] >= 0;
    }
    int upto = found;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int v = __shfl_up(upto, d);
        if (l >= d) upto += v;
    }
    if (l == 63) before[w] = upto;
    __syncthreads();
    int at = upto - found, n = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        if (i < w) at += before[i];
        n += before[i];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (mine[i] >= 0) list[at++] = ((int)threadIdx.x * kEach + i) << 16 | mine[i];
    __syncthreads();

    v4f acc[NT][TR];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < TR; ++r) acc[t][r] = v4f{0, 0, 0, 0};
    const int plane = a.T * a.K * a.F * U::kPlane;
    const __amdgpu_buffer_rsrc_t hs = rsrc(a.work + kPlanesAt, plane * P);
    const int units = (a.F + 4 * U::KL - 1) / (4 * U::KL), parts = (units + UN - 1) / UN;
    n = __builtin_amdgcn_readfirstlane(n);
    const int pieces = n * parts, place_k = (l >> 4) * U::KL;
    // a piece: UN units of a slot's rows of D, and lane t: the place of token t
    struct Piece {
        Units<KIND, TR, UN, WIDE> w;
        int place, u0;
    };
    auto load = [&](int q, Piece &p) {
        q = min(q, pieces - 1);  // past the last: it again, unused
        const int named = __builtin_amdgcn_readfirstlane(list[q / parts]);
        const int slot = named >> 16, e = named & 0xffff;
        p.place = reinterpret_cast<const uint8_t *>(a.work)[kMapAt + slot * kFewTokens + l];
        p.u0 = q % parts * UN;
        Rows<KIND, TR> down;
        down.init(a.down + e * a.out_block, a.down_scale + e * a.out_scale_block, n0, a.H, a.F);
        p.w.load(down, p.u0);
        issue();
    };
    Piece now, next;
    if (w < pieces) load(w, now);
    for (int q = w; q < pieces; q += NW) {
        // The slot's tokens take columns next to each other: lane c gets the entry of the
        // c-th, and lane t the column of token t.
        const uint64_t has = __ballot(now.place > 0);
        const int tokens = __popcll(has), below = __popcll(has & ((1ull << l) - 1));
        const int entry = __builtin_amdgcn_ds_permute((now.place > 0 ? below : tokens + l - below) * 4,
                                                      l * a.K + now.place - 1);
        const int column = now.place > 0 ? below : -1;
        v4f d[TR];
        auto clear = [&] {
#pragma unroll
            for (int r = 0; r < TR; ++r) d[r] = v4f{0, 0, 0, 0};
        };
        // Columns c0 .. c0 + 15, or fewer that lie `apart`, are added to their tokens' sums. Each
        // token takes its own alone: 0 times an infinite weight would be NaN.
        auto add = [&](int c0, int apart) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if ((has >> (t * 16) & 0xffff) == 0) continue;
                const int col = (__shfl(column, t * 16 + (l & 15)) - c0) * apart;
                const bool takes = col >= 0 && col < 16;
#pragma unroll
                for (int r = 0; r < TR; ++r)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float v = __shfl(d[r][j], (col & 15) | (l & 48));
                        acc[t][r][j] += takes ? v : 0.0f;
                    }
            }
        };
        clear();
        if (tokens <= kFewColumns) {
            Token<KIND, P, UN> x[kFewColumns];
#pragma unroll
            for (int c = 0; c < kFewColumns; ++c)
                if (c < tokens)
                    plane_fragment<KIND>(hs, __builtin_amdgcn_readlane(entry, c) * a.F * U::kPlane,
                                         Token<KIND, P, UN>::k_at(now.u0), a.F, plane, x[c].x);
            load(q + NW, next);
            tiles::each<UN>([&](auto at) {
                constexpr int i = decltype(at)::value;
                v4u f[P][U::J];
                x[0].template of_unit<i, -1>(f);
                tiles::each<kFewColumns - 1>([&](auto c) {
                    constexpr int C = decltype(c)::value + 1;
                    if (C < tokens) x[C].template of_unit<i, C>(f);
                });
#pragma unroll
                for (int r = 0; r < TR; ++r) d[r] = now.w.mma(r, i, f, d[r]);
            });
            add(0, 16 / kFewColumns);
        } else {
            auto group = [&](int c0, auto first) {
                const int e = __shfl(entry, c0 + (l & 15));
                const int row = c0 + (l & 15) < tokens ? e * a.F * U::kPlane : -1;
                // units at a time whose fragments are few registers
                constexpr int kAtOnce = P * U::J <= 3 ? UN : 1;
                tiles::each<UN / kAtOnce>([&](auto at) {
                    constexpr int i0 = decltype(at)::value * kAtOnce;
                    v4u x[kAtOnce][P][U::J];
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
                        for (int j = 0; j < U::J; ++j) {
                            v4u f[P];
                            plane_fragment<KIND>(hs, row, (now.u0 + i0 + i) * 4 * U::KL + place_k + j * 8, a.F,
                                                 plane, f);
#pragma unroll
                            for (int p = 0; p < P; ++p) x[i][p][j] = f[p];
                        }
                    if constexpr (decltype(first)::value && i0 == 0) load(q + NW, next);
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
                        for (int r = 0; r < TR; ++r) d[r] = now.w.mma(r, i0 + i, x[i], d[r]);
                });
                add(c0, 1);
            };
            group(0, std::true_type());
            for (int c0 = 16; c0 < tokens; c0 += 16) {
                clear();
                group(c0, std::false_type());
            }
        }
        now = next;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < TR; ++r) sums[w][t * TR + r][l] = acc[t][r];
    __syncthreads();
    for (int t = w; t < NT * TR; t += NW) {
        v4f v = sums[0][t][l];
#pragma unroll
        for (int i = 1; i < NW; ++i) v += sums[i][t][l];
        const int token = t / TR * 16 + (l & 15), col = n0 + t % TR * 16 + (l >> 4) * 4;
        if (token >= a.T || col >= a.H) continue;
        const int64_t to = (int64_t)token * a.H + col;
        const float f[4] = {v[0], v[1], v[2], v[3]};
        store_elems<4, U::kRow == 2, false>(a.out, to, f);
    }
}

template <int KIND, int NT, int TR, int UN, int NW, bool WIDE>
hipError_t few_in(const FewArgs &a, hipStream_t st) {
    hipLaunchKernelGGL((k_few_in<KIND, NT, TR, UN, NW, WIDE>), dim3((a.F + 16 * TR - 1) / (16 * TR), a.slots),
                       dim3(NW * 64), 0, st, a);
    return hipGetLastError();
}

template <int KIND, int NT, int TR, int UN, int NW, bool WIDE>
hipError_t few_out(const FewArgs &a, hipStream_t st) {
    hipLaunchKernelGGL((k_few_out<KIND, NT, TR, UN, NW, WIDE>), dim3((a.H + 16 * TR - 1) / (16 * TR)),
                       dim3(NW * 64), 0, st, a);
    return hipGetLastError();
}

// Waves of a workgroup and units of a load, us of the first kernel:
//   waves x units                          8 x 2    4 x 4    2 x 4     (4 bits)  8 x 4  4 x 4  2 x 4
//   1 token, 8 of 64, 2048 x 1024          15.8     17.5     17.1                                      bf16
//   64 tokens, 2 of 8, 4096 x 2048         64       67                           39.7   33.0   37.5
//   24 (4 bits: 8) tokens of 896 experts,
//   7168 x 512                             513      508      508                 120    92     80
//   64 tokens of 896 experts, 7168 x 512   954      933                          437    339    292
// Weights of 4 bits leave short rows, so the fewer waves share them the longer each loads.
template <int KIND, int NT, bool WIDE>
hipError_t few_in_of(const FewArgs &a, hipStream_t st) {
    if constexpr (!kScaled<KIND>) {
        return few_in<KIND, NT, 1, 2, 8, WIDE>(a, st);
    } else {
        constexpr int UN = KIND == kMxF32 ? 2 : 4;  // three pieces take the registers
        if ((int64_t)((a.F + 15) / 16) * a.slots > 1024) return few_in<KIND, NT, 1, UN, 2, WIDE>(a, st);
        return few_in<KIND, NT, 1, UN, 4, WIDE>(a, st);
    }
}

// Rows of D and waves of a workgroup, us of the second kernel (24 tokens, 8 in 4 bits, of 128
// experts, 8 each; 64 tokens of 8 experts, 2 each):
//   rows x waves                   16 x 4   16 x 8   16 x 16   32 x 4   32 x 8
//   24 tokens, 4096 x 512            83       68       121       98       89      bf16
//              4608 x 512           112      119       215       97       90
//   64 tokens, 4096 x 1024           41       37        55       50       44
//              4608 x 1024           64       68        99       50       44
//    8 tokens, 4096 x 512            22       19        71       29       39      4 bits
//              4608 x 512            31       33       103       29       39
//   64 tokens, 4096 x 1024           36      (33)                38       64
//              4608 x 1024           65      (59)                38       65
//   24 tokens, 4096 x 512           155      117       110      199      146      f32
//              4608 x 512           195      180       181      198      150
//   24 tokens, 4096 x 512            49       39                 56       46      f32, 4 bits
//              4608 x 512            64       68                 54       45
// A compute unit holds one workgroup, whose registers are many: 4096 columns in sixteens are one
// round of them, so past that 32 rows share the activations' loads between them (and at 3584,
// 5632 and 7168 columns too it is as at 4096 and 4608). In binary32 the matrix units are slow
// enough to want more waves. 8 waves leave 256 registers each, too few for 4 bits with many tokens
// or 32 rows (times in brackets are with some of them in scratch memory). One token of 8 experts of
// 2048 x 1024 in bf16 takes 13.5 us with 8 waves, 15.7 with 4 and 15.1 with 16.
template <int KIND, int NT, bool WIDE>
hipError_t few_out_of(const FewArgs &a, hipStream_t st) {
    constexpr int UN = KIND == kMxF32 ? 2 : 4;
    constexpr int kWide = KIND == kMxBf16 || (KIND == kMxF32 && NT == 4) ? 4 : 8;
    if (a.H > 4096) return few_out<KIND, NT, 2, UN, kWide, WIDE>(a, st);
    constexpr int NW = KIND == kF32 ? 16 : KIND == kMxBf16 && NT == 4 ? 4 : 8;
    return few_out<KIND, NT, 1, UN, NW, WIDE>(a, st);
}

template <int KIND, int NT>
hipError_t few_layer(const FewArgs &a, hipStream_t st) {
    hipError_t e;
    if constexpr (KIND == kMxBf16) {
        e = a.H % 512 == 0 ? few_in_of<KIND, NT, true>(a, st) : few_in_of<KIND, NT, false>(a, st);
        if (e != hipSuccess) return e;
        return a.F % 512 == 0 ? few_out_of<KIND, NT, true>(a, st) : few_out_of<KIND, NT, false>(a, st);
    } else {
        e = few_in_of<KIND, NT, false>(a, st);
        return e != hipSuccess ? e : few_out_of<KIND, NT, false>(a, st);
    }
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
