// A linear layer's weight and bias gradients from its input held in 8 bits
// (include/flashopt_lm.h): weight = dy^T x, the sum over the tokens.
//
// Mathematics.  A held value q 2^e has 7 bits: it is exact in BF16, and in FP16
// between that type's bounds of e.  So the matrix instructions of dy's own type
// take both factors exactly and sum in binary32.  A binary32 dy is three BF16
// numbers, its upper 8 bits, the next 8 and the last 8 (by truncation, so none
// overflows): three products in place of one, against the binary32 matrix
// instructions' 1/16 of the rate.  BF16's smallest step is 2^-133, so a dy below 2^-110 is
// taken towards zero to a multiple of it.  (A scale against that would have to be one for
// all tokens of a column, which takes another pass over dy, and costs its largest numbers.)
//
// Both factors lie in memory with the summed index (tokens) as their slow one, the
// instructions want it within a lane.  Tiles are kept in LDS as they lie, [token]
// [column], and ds_read_b64_tr_b16 transposes on the way to the registers: of a group
// of 16 lanes, lane l gives the address of 4 columns of token l / 4, and gets 4 tokens
// of column l.  Columns are swapped in units of 32 bytes by the token, so that
// 32 lanes' reads (4 tokens x 64 bytes) touch all banks once.
//
// The codes become values on their way into LDS, once a block, while the products of the
// stage before run (in each wave that reads them it would be four times the work), and
// every load of the loop is unconditional and a stage and more ahead: with the bounds
// checked word by word 8192 x 14336 x 4096 BF16 took 1842 us, so 880.  There the matrix pipes
// work 61 % of the time, the LDS 47 %, and the VALU issues 5.9 instructions for each
// product; what is left is the phases' dependence at two waves a SIMD.  (1090 to 1110
// TFLOP/s; the library's plain product of these sizes reaches 930, its best 1210.  Tried
// and slower: the halves of the codes' words in turns against their 8 % of bank
// conflicts 2 %, products and the rest by turns 4 %, higher priority during products 11 %, two
// stages of loads in registers: they spill.)  FP32 8192 x 4096 x 4096: 680 us, 1210 TFLOP/s
// of BF16 products.
#include "grad_plan.hpp"
#include "held.hpp"

namespace flashopt {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
#define LDS_SPACE __attribute__((address_space(3)))

// FN x FK fragments of 32 x 32 a wave, WN x WK waves for a tile, G such teams that
// share out a block's stages
template <int kType, int FN, int FK, int WN, int WK, int G>
struct GradTile {
    static constexpr int kThreads = WN * WK * kWave;                 // of a team
    static constexpr int BN = WN * FN * 32, BK = WK * FK * 32;
    static constexpr int kPlanes = kType == FLASHOPT_FP32 ? 3 : 1;
    static constexpr int kRowN = BN * 2, kRowK = BK * 2;             // bytes of a token's row in LDS
    static constexpr int kPlane = kTokens * kRowN;
    static constexpr int kStageBytes = kPlanes * kPlane + kTokens * kRowK;
    static constexpr int kLoadsN = kTokens * BN / 8 / kThreads;      // 8 columns of dy a time
    static constexpr int kLoadsK = kTokens * BK / 16 / kThreads;     // 16 codes a time
    // a wave's strip of outputs on their way to memory: 32 rows of 16 bits or 16 of 32
    static constexpr int kStrip = 32 * (FK * 32 * 2 + 16);
    static constexpr int kTeamBytes = 2 * kStageBytes > WN * WK * kStrip ? 2 * kStageBytes : WN * WK * kStrip;
    static constexpr int kLds = G * kTeamBytes;
    // a wave's sums on their way to another team's wave
    static constexpr int kSums = (FN * FK * 16 + 4) * kWave * 4;
    static_assert(G == 1 || G / 2 * WN * WK * kSums <= kLds, "half the teams' sums fit");
};

struct GradArgs {
    const void* dy;
    int64_t m, n, dy_stride;
    const int8_t* codes;
    const uint8_t* powers;
    int64_t k, ld;
    void* weight;
    int64_t weight_stride;
    void* bias;
    // the first `whole` tiles are a block's each, the rest are cut along the tokens
    uint32_t tn, tk, whole, splits;
    int64_t stages;                              // of all tokens
    float *part, *part_bias;                     // of a cut tile's piece: BN x BK, BN sums of dy
};

// Item t of `total`: XCDs (blocks go to the 8 of them by turns) get runs of items of
// their own.
__device__ __forceinline__ uint32_t run_of(uint32_t t, uint32_t total) {
    const uint32_t xcd = t % 8, q = total / 8, r = total % 8;
    return xcd * q + (xcd < r ? xcd : r) + t / 8;
}
// Tile u in columns of at most 8 tiles of n, so that neighbours share rows in an L2.
__device__ __forceinline__ void grad_tile_of(uint32_t u, uint32_t tn, uint32_t tk, uint32_t& n,
                                             uint32_t& k) {
    const uint32_t group = 8 * tk, g = u / group, in = u % group;
    const uint32_t high = tn - g * 8 < 8 ? tn - g * 8 : 8;
    n = g * 8 + in % high;
    k = in / high;
}

// 32 bytes of a token's row, as they are swapped: four rows' pairs of them lie in the
// four quarters of the banks (rows of 128 bytes do so in two halves by themselves).
template <int kRowBytes>
__device__ __forceinline__ int swapped(int slot, int token) {
    static_assert(kRowBytes == 128 || kRowBytes % 256 == 0, "whole halves of the banks");
    return slot ^ (kRowBytes == 128 ? token & 2 : (token & 3) << 1);
}

template <int kType>
__device__ __forceinline__ f32x16 product(s16x8 a, s16x8 b, f32x16 c) {
    if constexpr (kType == FLASHOPT_FP16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The sum of a fragment's eight values in a lane, by pairs.
template <int kType>
__device__ __forceinline__ float eight_of(s16x8 v) {
    const u32x4 w = __builtin_bit_cast(u32x4, v);
    constexpr int kAs = kType == FLASHOPT_FP16 ? FLASHOPT_FP16 : FLASHOPT_BF16;
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = Elem<kAs>::get(w, 2 * i) + Elem<kAs>::get(w, 2 * i + 1);
    return (x[0] + x[1]) + (x[2] + x[3]);
}

// Eight values of dy, in one BF16 or FP16 word or three words of BF16 parts.
template <int kType> struct DyWord;
template <> struct DyWord<FLASHOPT_BF16> { u32x4 w; };
template <> struct DyWord<FLASHOPT_FP16> { u32x4 w; };
template <> struct DyWord<FLASHOPT_FP32> { u32x4 w, v; };

// the upper 16 bits of two numbers
__device__ __forceinline__ uint32_t halves(uint32_t lo, uint32_t hi) {
    return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

// x = hi + mid + low, each the upper 16 bits of its word (less what lies below 2^-133).  An
// infinity is its own hi (a NaN may be one there, but then mid is NaN).
__device__ __forceinline__ void three_parts(uint32_t x, uint32_t& hi, uint32_t& mid, uint32_t& low) {
    constexpr int kInfinities = 0x204;           // of v_cmp_class: -inf, +inf
    hi = x;
    const float r = __builtin_amdgcn_classf(as_f32(x), kInfinities) ? 0.0f : as_f32(x) - as_f32(x & 0xFFFF0000u);
    mid = as_u32(r);
    low = as_u32(r - as_f32(mid & 0xFFFF0000u));
}

// kBias: with the bias, added up from the fragments by the waves of the first columns
template <int kType, int FN, int FK, int WN, int WK, int G, bool kBias>
__global__ __launch_bounds__(G * WN * WK * kWave, 2) void weight_grad_kernel(GradArgs a) {
    typedef GradTile<kType, FN, FK, WN, WK, G> S;
    typedef typename Elem<kType>::T T;
    constexpr int P = S::kPlanes;
    extern __shared__ __attribute__((aligned(16))) int8_t all_lds[];
    const int team = G == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / S::kThreads);
    const int tid = G == 1 ? threadIdx.x : threadIdx.x % S::kThreads, lane = tid & (kWave - 1), wave = tid / kWave;
    const int wn = wave % WN, wk = wave / WN;
    int8_t* lds = all_lds + team * S::kTeamBytes;
    uint32_t in, ik;
    const bool cut = blockIdx.x >= a.whole;
    const uint32_t piece = cut ? run_of(blockIdx.x - a.whole, gridDim.x - a.whole) : 0;
    grad_tile_of(cut ? a.whole + piece / a.splits : run_of(blockIdx.x, a.whole), a.tn, a.tk, in, ik);
    const uint32_t split = piece % a.splits, splits = cut ? a.splits : 1;
    const int64_t n0 = (int64_t)in * S::BN, k0 = (int64_t)ik * S::BK;
    const int64_t parts = (int64_t)splits * G, part_of = (int64_t)split * G + team;
    const int64_t from = a.stages * part_of / parts, to = a.stages * (part_of + 1) / parts;
    const int64_t groups = a.ld / kGroup8;

    // ---- what is loaded: this thread's words of a stage, zeros behind the last token
    const T* dy = (const T*)a.dy + n0;
    const int8_t* codes = a.codes + k0;
    const uint8_t* powers = a.powers + k0 / kGroup8;
    const int64_t left_n = a.n - n0, left_k = a.ld - k0;
    DyWord<kType> g[S::kLoadsN];
    u32x4 q[S::kLoadsK];
    uint32_t byte[S::kLoadsK];
    constexpr int kWordsN = S::BN / 8, kWordsK = S::BK / 16;
    // Behind the last column the last words are read again: what comes of them is not
    // stored.  A word that begins before dy's last column and ends behind it reads the row's
    // neighbours, which are there except behind the last rows.
    const T* dy_at[S::kLoadsN];
    const int8_t* codes_at[S::kLoadsK];
    const uint8_t* powers_at[S::kLoadsK];
#pragma unroll
    for (int i = 0; i < S::kLoadsN; ++i) {
        const int w = i * S::kThreads + tid, c = w % kWordsN, last = (int)((left_n < S::BN ? left_n : S::BN) - 1) / 8;
        dy_at[i] = dy + (from * kTokens + w / kWordsN) * a.dy_stride + min(c, last) * 8;
    }
#pragma unroll
    for (int i = 0; i < S::kLoadsK; ++i) {
        const int w = i * S::kThreads + tid, c = w % kWordsK, last = (int)((left_k < S::BK ? left_k : S::BK) - 1) / 16;
        const int64_t t = from * kTokens + w / kWordsK;
        codes_at[i] = codes + t * a.ld + min(c, last) * 16;
        powers_at[i] = powers + t * groups + min(c, last) / 2;
    }
    const int64_t step_n = kTokens * a.dy_stride, step_k = kTokens * a.ld, step_p = kTokens * groups;
    auto advance = [&]() {
#pragma unroll
        for (int i = 0; i < S::kLoadsN; ++i) dy_at[i] += step_n;
#pragma unroll
        for (int i = 0; i < S::kLoadsK; ++i) codes_at[i] += step_k, powers_at[i] += step_p;
    };
    auto fetch = [&]() {                         // the next stage, all of it there
#pragma unroll
        for (int i = 0; i < S::kLoadsN; ++i) {
            const u32x4_any* v = reinterpret_cast<const u32x4_any*>(dy_at[i]);
            g[i].w = v[0];
            if constexpr (P == 3) g[i].v = v[1];
        }
#pragma unroll
        for (int i = 0; i < S::kLoadsK; ++i) {
            q[i] = *reinterpret_cast<const u32x4*>(codes_at[i]);
            byte[i] = *powers_at[i];
        }
        advance();
    };
    auto fetch_last = [&](int64_t stage) {       // one that may reach behind the last token
#pragma unroll
        for (int i = 0; i < S::kLoadsN; ++i) {
            const int w = i * S::kThreads + tid, c = w % kWordsN;
            constexpr int W = 8 / Elem<kType>::kE;
            const int64_t n = stage * kTokens + w / kWordsN < a.m ? left_n : 0;
            const T* p = dy + (n ? stage * kTokens + w / kWordsN : 0) * a.dy_stride;
            g[i].w = load_vec<kType>(p, c * W, n, 0);
            if constexpr (P == 3) g[i].v = load_vec<kType>(p, c * W + 1, n, 0);
        }
#pragma unroll
        for (int i = 0; i < S::kLoadsK; ++i) {
            const int w = i * S::kThreads + tid;
            q[i] = u32x4{0, 0, 0, 0};
            byte[i] = 0;
            if (stage * kTokens + w / kWordsK < a.m) {
                q[i] = *reinterpret_cast<const u32x4*>(codes_at[i]);
                byte[i] = *powers_at[i];
            }
        }
        advance();
    };
    // ---- into LDS, the codes as values
    auto put = [&](int half) {
        int8_t* d = lds + half * S::kStageBytes;
#pragma unroll
        for (int i = 0; i < S::kLoadsN; ++i) {
            const int w = i * S::kThreads + tid, c = w % kWordsN, t = w / kWordsN;
            int8_t* at = d + t * S::kRowN + swapped<S::kRowN>(c >> 1, t) * 32 + (c & 1) * 16;
            if constexpr (P == 1) {
                *(u32x4*)at = g[i].w;
            } else {
                u32x4 part[3];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t x0 = e < 2 ? g[i].w[2 * e] : g[i].v[2 * e - 4];
                    const uint32_t x1 = e < 2 ? g[i].w[2 * e + 1] : g[i].v[2 * e - 3];
                    uint32_t h0, m0, l0, h1, m1, l1;
                    three_parts(x0, h0, m0, l0);
                    three_parts(x1, h1, m1, l1);
                    part[0][e] = halves(h0, h1);
                    part[1][e] = halves(m0, m1);
                    part[2][e] = halves(l0, l1);
                }
#pragma unroll
                for (int p = 0; p < 3; ++p) *(u32x4*)(at + p * S::kPlane) = part[p];
            }
        }
        d += P * S::kPlane;
#pragma unroll
        for (int i = 0; i < S::kLoadsK; ++i) {
            const int w = i * S::kThreads + tid, c = w % kWordsK, t = w / kWordsK;
            const float up = as_f32(byte[i] << 23);
            u32x4 v[2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x[4];
                held_values(q[i][e], up, x);
                if constexpr (kType == FLASHOPT_FP16) {
                    v[e / 2][e % 2 * 2] = f32_to_f16(x[0]) | f32_to_f16(x[1]) << 16;
                    v[e / 2][e % 2 * 2 + 1] = f32_to_f16(x[2]) | f32_to_f16(x[3]) << 16;
                } else {
                    v[e / 2][e % 2 * 2] = halves(as_u32(x[0]), as_u32(x[1]));
                    v[e / 2][e % 2 * 2 + 1] = halves(as_u32(x[2]), as_u32(x[3]));
                }
            }
            int8_t* at = d + t * S::kRowK + swapped<S::kRowK>(c, t) * 32;
            *(u32x4*)at = v[0];
            *(u32x4*)(at + 16) = v[1];
        }
    };
    // ---- fragments: 32 columns x 16 tokens, lane l of column l % 32 with tokens
    // 4 (l / 32) + 0 .. 3 and the same 8 further
    const int sub = lane >> 4 & 1, token = 4 * (lane >> 5) + (lane & 15) / 4, eight = (lane & 3) * 8;
    auto read = [&](const int8_t* d, auto row, int slot, int step) {
        constexpr int kRow = decltype(row)::value;
        s16x4 r[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t = step * 16 + h * 8 + token;
            r[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (LDS_SPACE s16x4*)(d + t * kRow + swapped<kRow>(slot + sub, t) * 32 + eight));
        }
        return __builtin_shufflevector(r[0], r[1], 0, 1, 2, 3, 4, 5, 6, 7);
    };
    f32x16 acc[FK][FN];
    float sums[FN];                              // of this lane's tokens of dy
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        sums[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < FK; ++i) acc[i][j] = f32x16{};
    }
    const bool bias_here = kBias && ik == 0 && wk == 0;
    // A stage's products in phases: of its two steps of 16 tokens and, where registers are
    // few, of dy's parts, the small ones first.  A phase's fragments are read while the
    // one before it multiplies.
    constexpr int A = FK == 4 ? 1 : P, kPhases = 2 * P / A;          // parts of a phase
    s16x8 fx[2][FK], fy[2][A][FN];
    auto read_phase = [&](int q, int half) {
        const int8_t* d = lds + half * S::kStageBytes;
        const int step = q * A / P, first = P - A - q * A % P;
#pragma unroll
        for (int p = 0; p < A; ++p)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                fy[q & 1][p][j] = read(d + (first + p) * S::kPlane, std::integral_constant<int, S::kRowN>(), (wn * FN + j) * 2, step);
        if (q * A % P == 0)
#pragma unroll
            for (int i = 0; i < FK; ++i)
                fx[step][i] = read(d + P * S::kPlane, std::integral_constant<int, S::kRowK>(), (wk * FK + i) * 2, step);
    };
    auto products = [&](int q) {
#pragma unroll
        for (int p = A - 1; p >= 0; --p) {
#pragma unroll
            for (int i = 0; i < FK; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = product<kType>(fx[q * A / P][i], fy[q & 1][p][j], acc[i][j]);
            if (kBias && bias_here)
#pragma unroll
                for (int j = 0; j < FN; ++j) sums[j] += eight_of<kType>(fy[q & 1][p][j]);
        }
    };

    // A stage in LDS, the next one in registers on its way there, the one after that on its
    // way from memory.  Stages up to `whole` need no checks.
    {
        const int64_t sure = left_n >= S::BN || left_n % 8 == 0 ? a.m : a.m - 7;
        const int64_t whole = sure < 0 ? 0 : sure / kTokens;
        const int64_t last = G == 1 ? to : from + (a.stages + parts - 1) / parts;
        auto fetch_any = [&](int64_t s) {
            if (s >= to) return;
            if (s < whole) fetch();
            else fetch_last(s);
        };
        fetch_any(from);
        if (from < to) put(0);
        fetch_any(from + 1);
        __syncthreads();
        if (from < to) read_phase(0, 0);
        int64_t s = from;
        int half = 0;
        for (; s + 2 < to && s + 2 < whole; ++s, half ^= 1) {
            read_phase(1, half);
            products(0);
            put(half ^ 1);
            fetch();
#pragma unroll
            for (int q = 1; q < kPhases - 1; ++q) {
                read_phase(q + 1, half);
                products(q);
            }
            __syncthreads();
            read_phase(0, half ^ 1);
            products(kPhases - 1);
        }
        for (; s < last; ++s, half ^= 1) {       // every team meets the same number of barriers
            if (s < to) {
                read_phase(1, half);
                products(0);
                if (s + 1 < to) put(half ^ 1);
                fetch_any(s + 2);
#pragma unroll
                for (int q = 1; q < kPhases - 1; ++q) {
                    read_phase(q + 1, half);
                    products(q);
                }
            }
            __syncthreads();
            if (s < to) {
                if (s + 1 < to) read_phase(0, half ^ 1);
                products(kPhases - 1);
            }
        }
        __syncthreads();
    }
    // The teams' sums: the upper half's to the lower half's waves, until one team has all.
    if constexpr (G > 1) {
#pragma unroll
        for (int h = G / 2; h >= 1; h /= 2) {
            if (team >= h && team < 2 * h) {
                int8_t* d = all_lds + ((team - h) * WN * WK + wave) * S::kSums + lane * 16;
#pragma unroll
                for (int i = 0; i < FK; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const f32x16 c = acc[i][j];
                            *(u32x4*)(d + ((i * FN + j) * 4 + b) * kWave * 16) = u32x4{as_u32(c[4 * b]), as_u32(c[4 * b + 1]), as_u32(c[4 * b + 2]), as_u32(c[4 * b + 3])};
                        }
                if (kBias)
#pragma unroll
                    for (int j = 0; j < FN; ++j) *(float*)(d + FN * FK * 4 * kWave * 16 + j * 4) = sums[j];
            }
            __syncthreads();
            if (team < h) {
                const int8_t* d = all_lds + (team * WN * WK + wave) * S::kSums + lane * 16;
#pragma unroll
                for (int i = 0; i < FK; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const u32x4 v = *(const u32x4*)(d + ((i * FN + j) * 4 + b) * kWave * 16);
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[i][j][4 * b + e] += as_f32(v[e]);
                        }
                if (kBias)
#pragma unroll
                    for (int j = 0; j < FN; ++j) sums[j] += *(const float*)(d + FN * FK * 4 * kWave * 16 + j * 4);
            }
            __syncthreads();
        }
        if (team != 0) return;
    }
    static_assert(FN <= 4, "a lane's bias sums in 16 bytes");
    static_assert(kTokens == 32, "two steps a stage");

    // ---- outputs.  A fragment's column (lane) is an n, its rows are k: register r
    // holds k = 8 (r / 4) + 4 (lane / 32) + r % 4.
    const int64_t nw = n0 + wn * FN * 32, kw = k0 + wk * FK * 32;
    if (kBias && bias_here) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int64_t n = nw + j * 32 + lane;
            const float x = sums[j] + __shfl_xor(sums[j], 32);
            if (lane >= 32) continue;
            if (cut) a.part_bias[(int64_t)piece * S::BN + (n - n0)] = x;
            else if (n < a.n) ((T*)a.bias)[n] = Elem<kType>::down(x);
        }
    }
    // Through LDS, 16 or 32 outputs of n at a time, so that rows are written in whole words.
    // (Only this wave's own strip: LDS keeps a wave's accesses in order.)
    int8_t* strip = lds + wave * S::kStrip;
    auto write = [&](auto type, auto store) {
        constexpr int kOut = decltype(type)::value, kEach = kOut == FLASHOPT_FP32 ? 4 : 2;
        constexpr int kRows = kEach == 4 ? 16 : 32, kStride = FK * 32 * kEach + 16;
        constexpr int kWords = FK * 32 * kEach / 16;
        static_assert(kRows * kStride <= S::kStrip, "the strip fits");
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int h = 0; h < 32 / kRows; ++h) {
                const int r = (lane & 31) - h * kRows;
                if (r >= 0 && r < kRows) {
#pragma unroll
                    for (int i = 0; i < FK; ++i)
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            int8_t* at = strip + r * kStride + (i * 32 + b * 8 + 4 * (lane >> 5)) * kEach;
                            const f32x16 c = acc[i][j];
                            if constexpr (kEach == 4) {
                                *(u32x4*)at = u32x4{as_u32(c[4 * b]), as_u32(c[4 * b + 1]), as_u32(c[4 * b + 2]), as_u32(c[4 * b + 3])};
                            } else {
                                const float y[8] = {c[4 * b], c[4 * b + 1], c[4 * b + 2], c[4 * b + 3], 0.0f, 0.0f, 0.0f, 0.0f};
                                const u32x4 v = pack<kOut>(y);
                                *(u32x2*)at = u32x2{v[0], v[1]};
                            }
                        }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int w = lane; w < kRows * kWords; w += kWave) {
                    const int row = w / kWords, word = w % kWords;
                    store(wn * FN * 32 + j * 32 + h * kRows + row, word, *(const u32x4*)(strip + row * kStride + word * 16));
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
    };
    if (cut) {
        uint32_t* part = (uint32_t*)a.part + (int64_t)piece * (S::BN * S::BK) + wk * FK * 32;
        write(std::integral_constant<int, FLASHOPT_FP32>(), [&](int row, int word, const u32x4& v) {
            *(u32x4*)(part + row * S::BK + word * 4) = v;
        });
    } else {
        T* out = (T*)a.weight + n0 * a.weight_stride + kw;
        write(std::integral_constant<int, kType>(), [&](int row, int word, const u32x4& v) {
            if (n0 + row < a.n && kw < a.k) store_vec<kType>(out + row * a.weight_stride, word, a.k - kw, v);
        });
    }
}

// A cut tile's pieces added in order, a word of outputs a thread.
template <int kType, int BN, int BK>
__global__ __launch_bounds__(kBlock) void weight_grad_join_kernel(GradArgs a, bool bias) {
    typedef typename Elem<kType>::T T;
    constexpr int E = Elem<kType>::kE, kWords = BK / E, kBlocks = BN * kWords / kBlock;
    const uint32_t tile = blockIdx.x / kBlocks;
    uint32_t in, ik;
    grad_tile_of(a.whole + tile, a.tn, a.tk, in, ik);
    const int at = blockIdx.x % kBlocks * kBlock + threadIdx.x, row = at / kWords, w = at % kWords;
    const int64_t n0 = (int64_t)in * BN, k0 = (int64_t)ik * BK;
    if (n0 + row < a.n && k0 + w * E < a.k) {
        const uint32_t* p = (const uint32_t*)a.part + (int64_t)tile * a.splits * (BN * BK) + row * BK + w * E;
        float x[E] = {};
#pragma unroll 4
        for (uint32_t s = 0; s < a.splits; ++s, p += BN * BK)
#pragma unroll
            for (int h = 0; h < E / 4; ++h) {
                const u32x4 v = *(const u32x4*)(p + 4 * h);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * h + e] += as_f32(v[e]);
            }
        store_vec<kType>((T*)a.weight + (n0 + row) * a.weight_stride + k0, w, a.k - k0, pack<kType>(x));
    }
    if (bias && ik == 0 && w == 0 && n0 + row < a.n) {
        float x = 0.0f;
        for (uint32_t s = 0; s < a.splits; ++s) x += a.part_bias[((int64_t)tile * a.splits + s) * BN + row];
        ((T*)a.bias)[n0 + row] = Elem<kType>::down(x);
    }
}

// ---- host ---------------------------------------------------------------------

template <typename F>
static int by_type(int32_t type, F f) {
    if (type == FLASHOPT_BF16) f(std::integral_constant<int, FLASHOPT_BF16>());
    else if (type == FLASHOPT_FP16) f(std::integral_constant<int, FLASHOPT_FP16>());
    else f(std::integral_constant<int, FLASHOPT_FP32>());
    return launch_status();
}

template <int kType, int FN, int FK, int WN, int WK, int G, bool kBias>
static void launch_grad(const GradArgs& a, hipStream_t st) {
    typedef GradTile<kType, FN, FK, WN, WK, G> S;
    const uint32_t cut = a.tn * a.tk - a.whole;
    hipLaunchKernelGGL((weight_grad_kernel<kType, FN, FK, WN, WK, G, kBias>), dim3(a.whole + cut * a.splits),
                       dim3(G * S::kThreads), S::kLds, st, a);
    if (cut)
        hipLaunchKernelGGL((weight_grad_join_kernel<kType, S::BN, S::BK>),
                           dim3(cut * (S::BN * S::BK / Elem<kType>::kE / kBlock)), dim3(kBlock), 0, st, a, kBias);
}

static int check_grad_shape(int32_t type, int64_t m, int64_t n, int64_t k) {
    if (!valid_type(type)) return FLASHOPT_ERR_ARG;
    const int64_t most = int64_t(1) << 24;
    // a launch has less than 2^32 threads
    if (m < 0 || m > most || n < 0 || n > most || k < 1 || k > FLASHOPT_INT8_COLS_MAX ||
        (n / 128 + 1) * (k / 128 + 1) > most / 2)
        return FLASHOPT_ERR_SIZE;
    return FLASHOPT_OK;
}

}  // namespace flashopt

using namespace flashopt;

extern "C" {

size_t flashopt_held_weight_grad_workspace_bytes(int32_t type, int64_t m, int64_t n, int64_t k) {
    if (check_grad_shape(type, m, n, k) || n == 0) return 0;
    const GradPlan p = grad_plan(type, m, n, held_ld(k), true);
    return p.part + p.bias;
}

int flashopt_held_weight_grad(const void* dy, int32_t type, int64_t m, int64_t n,
                              int64_t dy_stride, const int8_t* codes, const uint8_t* powers,
                              int64_t k, void* weight, int64_t weight_stride, void* bias,
                              void* workspace, size_t workspace_bytes, void* stream) {
    const int e = check_grad_shape(type, m, n, k);
    if (e) return e;
    if (dy_stride < n || dy_stride > kMaxNumel || weight_stride < k || weight_stride > kMaxNumel)
        return FLASHOPT_ERR_SIZE;
    if (n == 0) return FLASHOPT_OK;
    const size_t size = type_size(type);
    if (!weight || (m > 0 && (!dy || !codes || !powers))) return FLASHOPT_ERR_NULL;
    if (!aligned(weight, size) || !aligned(bias, size) || !aligned(dy, size) || !aligned(codes, 16))
        return FLASHOPT_ERR_ALIGN;
    // (as spans: their rows are of other kinds)
    if (m > 0) {
        const uintptr_t d0 = (uintptr_t)dy, w0 = (uintptr_t)weight;
        const __int128 d1 = (__int128)d0 + ((__int128)(m - 1) * dy_stride + n) * size;
        const __int128 w1 = (__int128)w0 + ((__int128)(n - 1) * weight_stride + k) * size;
        if ((__int128)d0 < w1 && (__int128)w0 < d1) return FLASHOPT_ERR_ARG;
    }
    const int64_t each = (int64_t)size, held = m * held_ld(k);
    const __int128 row = (__int128)weight_stride * each;
    if (rows_meet(n, weight, row, k * each, codes, held) || rows_meet(n, weight, row, k * each, powers, held / kGroup8) ||
        rows_meet(n, weight, row, k * each, bias, n * each) || rows_meet(m, dy, (__int128)dy_stride * each, n * each, bias, n * each) ||
        rows_meet(1, bias, 0, n * each, codes, held) || rows_meet(1, bias, 0, n * each, powers, held / kGroup8))
        return FLASHOPT_ERR_ARG;
    const GradPlan p = grad_plan(type, m, n, held_ld(k), bias != nullptr);
    if (p.part + p.bias) {
        if (!workspace) return FLASHOPT_ERR_NULL;
        if (workspace_bytes < p.part + p.bias || !aligned(workspace, 256)) return FLASHOPT_ERR_WORKSPACE;
    }
    const GradArgs a = {dy, m, n, dy_stride, codes, powers, k, held_ld(k), weight, weight_stride, bias,
                        (uint32_t)p.tn, (uint32_t)p.tk, (uint32_t)p.whole, (uint32_t)p.splits,
                        (m + kTokens - 1) / kTokens, (float*)workspace,
                        (float*)((char*)workspace + p.part)};
    const hipStream_t st = (hipStream_t)stream;
    return by_type(type, [&](auto t) {
        constexpr int kType = decltype(t)::value;
        constexpr int kTeamsOf = kType == FLASHOPT_FP32 ? 2 : 4, kHigh = kType == FLASHOPT_FP32 ? 2 : 4;
        if (p.way == GradPlan::kLarge) {
            if (bias) launch_grad<kType, 2, 4, kHigh, 2, 1, true>(a, st);
            else launch_grad<kType, 2, 4, kHigh, 2, 1, false>(a, st);
        } else if (p.way == GradPlan::kTeams) {
            if (bias) launch_grad<kType, 1, 2, 2, 2, kTeamsOf, true>(a, st);
            else launch_grad<kType, 1, 2, 2, 2, kTeamsOf, false>(a, st);
        } else {
            if (bias) launch_grad<kType, 2, 2, 2, 2, 1, true>(a, st);
            else launch_grad<kType, 2, 2, 2, 2, 1, false>(a, st);
        }
    });
}

}  // extern "C"
