// Rows in 8 bits and the linear layer over them (include/flashopt_lm.h).
//
// Mathematics.  A row x with a = max |x_c| is held as q_c = rne(127 x_c / a)
// and the scale a / 127.  For rows a_i of tokens and b_j of output channels,
//   y_ij = s_i w_j sum_c q_ic v_jc + bias_j:
// the sum runs in integers (v_mfma_i32_*_i8), exactly, since at most 2^17
// products of at most 127^2 stay below 2^31; the scales enter once, at the
// end, in binary32.
#include <cmath>

#include "rows.hpp"

namespace flashopt {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int64_t kLdStep = 128;
static inline int64_t ld_of(int64_t cols) { return (cols + kLdStep - 1) / kLdStep * kLdStep; }

// ---- rounding a row -----------------------------------------------------------

// rne(127 x / a), decided as by exact division.  r = RN(127 / a): x r is within
// 2^-22 of the quotient relative to it, below 2^-15 absolutely, so only a value
// that lies within 2^-14 of a border between two codes needs more: there the
// quotient is formed in binary64, whose rounding error (2^-46 at most here)
// moves it over no border unless an FP32 row holds a value that close to one.
__device__ __forceinline__ int row_code(float x, float a, float r) {
    const float v = x * r;
    float q = __builtin_rintf(v);
    if (__builtin_fabsf(v - q) > 0.5f - 0x1p-14f) q = (float)__builtin_rint((double)x * 127.0 / (double)a);
    return (int)fminf(fmaxf(q, -127.0f), 127.0f);
}

// A row's largest magnitude, as a pattern: infinities and NaN rank above all.
struct RowScale {
    float a, r;
    bool bad, small;
    __device__ __forceinline__ explicit RowScale(uint32_t top) : a(as_f32(top)) {
        bad = top >= 0x7F800000u;
        // below 2^-100, 127 / a overflows or x r is of a subnormal: binary64 for all
        small = a < 0x1p-100f;
        r = small || bad ? 0.0f : 127.0f / a;
    }
    __device__ __forceinline__ int code(float x) const {
        if (bad || a == 0.0f) return 0;
        return small ? (int)__builtin_rint((double)x * 127.0 / (double)a) : row_code(x, a, r);
    }
    __device__ __forceinline__ float scale() const { return bad ? NAN : a / 127.0f; }
};

// the largest of a block's patterns; red: one word per wave
template <int kWaves>
__device__ __forceinline__ uint32_t block_max(uint32_t top, uint32_t* red) {
    top = wave_max_u32(top);
    if (kWaves == 1) return top;
    if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = max(top, red[w]);
    return top;
}

// The codes of one 16-byte word, from entry j of its row on; entries past the
// row are 0.
template <int kType>
__device__ __forceinline__ void word_codes(const u32x4& v, int64_t j, int64_t cols,
                                           const RowScale& S, int8_t* out) {
    constexpr int E = Elem<kType>::kE;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int q = j + e < cols ? S.code(Elem<kType>::get(v, e)) : 0;
        w[e / 4] |= ((uint32_t)q & 0xFFu) << (8 * (e % 4));
    }
    if (E == 8) *reinterpret_cast<u32x2*>(out + j) = u32x2{w[0], w[1]};
    else *reinterpret_cast<uint32_t*>(out + j) = w[0];
}

// One block of kWaves waves per row, the row in registers: read once.
// 8192 rows of 4096 in BF16: 24 us, 4.2 TB/s; element by element in two passes 80.
template <int kType, int kWaves, int kVecs>
__global__ __launch_bounds__(kWaves * kWave) void quantize_rows_kernel(
    const typename Elem<kType>::T* x, int64_t cols, int64_t stride, int64_t ld, int8_t* codes,
    float* scale, int64_t first) {
    constexpr int E = Elem<kType>::kE;
    __shared__ uint32_t red[kWaves];
    const int64_t row = first + blockIdx.x;
    const typename Elem<kType>::T* p = x + row * stride;
    u32x4 r[kVecs];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) r[i] = load_vec<kType>(p, i * kWaves * kWave + threadIdx.x, cols, 0);
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) top = max(top, as_u32(Elem<kType>::get(r[i], e)) & 0x7FFFFFFFu);
    const RowScale S(block_max<kWaves>(top, red));
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int64_t j = ((int64_t)i * kWaves * kWave + threadIdx.x) * E;
        if (j < ld) word_codes<kType>(r[i], j, cols, S, codes + row * ld);
    }
    if (threadIdx.x == 0) scale[row] = S.scale();
}

// Longer rows: read twice.
template <int kType>
__global__ __launch_bounds__(kBlock) void quantize_long_kernel(const typename Elem<kType>::T* x,
                                                               int64_t cols, int64_t stride,
                                                               int64_t ld, int8_t* codes,
                                                               float* scale, int64_t first) {
    constexpr int E = Elem<kType>::kE;
    __shared__ uint32_t red[kWavesPerBlock];
    const int64_t row = first + blockIdx.x;
    const typename Elem<kType>::T* p = x + row * stride;
    uint32_t top = 0;
    for (int64_t w = threadIdx.x; w * E < cols; w += kBlock) {
        const u32x4 v = load_vec<kType>(p, w, cols, 0);
#pragma unroll
        for (int e = 0; e < E; ++e) top = max(top, as_u32(Elem<kType>::get(v, e)) & 0x7FFFFFFFu);
    }
    const RowScale S(block_max<kWavesPerBlock>(top, red));
    for (int64_t w = threadIdx.x; w * E < ld; w += kBlock)
        word_codes<kType>(load_vec<kType>(p, w, cols, 0), w * E, cols, S, codes + row * ld);
    if (threadIdx.x == 0) scale[row] = S.scale();
}

// The same from a tensor's state: the rebuilt master weight, element by
// element and twice (an export; rows start at any element of the state's blocks).
// 14336 x 4096 of AdamW: 114 us, bound by its scalar loads; the bytes take 46 at the
// rate of a copy.
template <int kOpt, bool kFp32>
__global__ __launch_bounds__(kBlock) void quantize_state_kernel(DevTensor d, int64_t cols,
                                                                int64_t ld, int8_t* codes,
                                                                float* scale, int64_t first) {
    const int64_t row = first + blockIdx.x;
    const GTensor T = view(d);
    auto load = [&](int64_t j) -> float {
        const int64_t e = row * cols + j;
        if (kFp32) {
            constexpr int F = kOpt == kAdamW ? 3 : 2;
            return ((const GLOBAL float*)T.codes)[(e >> 9) * (512 * F) + (e & 511)];
        }
        return unsplit(T.theta[e], (int32_t)(int8_t)*code_at<kOpt>(T, e, kRho));
    };
    __shared__ uint32_t red[kWavesPerBlock];
    uint32_t top = 0;
    for (int64_t j = threadIdx.x; j < cols; j += kBlock) top = max(top, as_u32(load(j)) & 0x7FFFFFFFu);
    const RowScale S(block_max<kWavesPerBlock>(top, red));
    for (int64_t j = threadIdx.x; j < ld; j += kBlock)
        codes[row * ld + j] = (int8_t)(j < cols ? S.code(load(j)) : 0);
    if (threadIdx.x == 0) scale[row] = S.scale();
}

// ---- the product: tiles -----------------------------------------------------------

// A block computes BN output channels x BM tokens with WN x WM waves, each FN x
// FM products of v_mfma_i32_32x32x32_i8 (the weight rows as A, the tokens as
// B: lane l holds 16 codes of row l % 32; afterwards, of token l % 32, the
// channels 8 (r / 4) + 4 (l / 32) + r % 4).  Stages of 128 codes (one line of
// each row) go global -> registers -> LDS, two in LDS, in four steps of 32 codes:
//   step 0, 1: half of the next stage's registers each go to its LDS half,
//   step 1, 2: and the loads of the stage after it are issued into them;
//   barrier:   the next stage is written, this one read;
//   step 3:    the next stage's first fragments are read.
// Each step reads the next step's fragments, and its products are spread over
// what it issues (sched_group_barrier).  A row of 128 bytes keeps its word c
// at c ^ (row / 2 & 7): the 16 rows read at a time, or the two rows of 8 words
// written, lie in all 64 banks.
//
// Blocks stay and take tile after tile; the stages run on over a tile's end,
// so that the next tile's first stages are loaded while this one's last
// products and its output are under way.
//
// kSplit: where there are few tiles, each is cut along the row into `splits`
// pieces that count as tiles here; a piece's integer sums go to `sums` as the
// registers hold them, 16 bytes of each lane after the other's, and
// join_kernel adds them up and writes the output.
constexpr int kStage = 128;

template <int kType, int FN, int FM, int WN, int WM>
struct Tile {
    static constexpr int kThreads = WN * WM * kWave;
    static constexpr int BN = WN * FN * 32, BM = WM * FM * 32;
    static constexpr int kStageBytes = (BN + BM) * kStage;
    static constexpr int kLoads = kStageBytes / 16 / kThreads;
    static constexpr int kRowsPerLoad = kThreads / 8;
    // a tile's scales and bias: BN weight scales, BN biases, BM token scales
    static constexpr int kScales = 2 * BN + BM, kScalesEach = (kScales + kThreads - 1) / kThreads;
    static constexpr int kPlace = kScalesEach * kThreads;
    static constexpr size_t kLds = 2 * kStageBytes + 2 * kPlace * sizeof(float);
    // blocks that a CU holds (160 KB of LDS)
    static constexpr int kBlocks = kLds > 80 * 1024 ? 1 : 2;
};

// Tile t of the order in which blocks take them.  Blocks go to the 8 XCDs by
// turns; each XCD gets a run of tiles of its own, ordered in columns of at
// most 8 token tiles, so that the tiles an XCD works on at a time share rows in
// its L2.
__device__ __forceinline__ void tile_of(uint32_t t, uint32_t tn, uint32_t tm, uint32_t& n,
                                        uint32_t& m) {
    const uint32_t total = tn * tm, xcd = t % 8, k = t / 8;
    const uint32_t q = total / 8, r = total % 8;
    const uint32_t u = xcd * q + (xcd < r ? xcd : r) + k;
    const uint32_t group = 8 * tn, g = u / group, in = u % group;
    const uint32_t high = tm - g * 8 < 8 ? tm - g * 8 : 8;
    m = g * 8 + in % high;
    n = in / high;
}

// four values rounded to a 16-bit type
template <int kType>
__device__ __forceinline__ u32x2 pack4(const float* y) {
    const float z[8] = {y[0], y[1], y[2], y[3], 0.0f, 0.0f, 0.0f, 0.0f};
    const u32x4 v = pack<kType>(z);
    return u32x2{v[0], v[1]};
}

template <int kType, int FN, int FM, int WN, int WM, bool kSplit>
__global__ __launch_bounds__(WN * WM * kWave, 2) void tile_kernel(
    const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale,
    const typename Elem<kType>::T* bias, int64_t m, int64_t n, int32_t ld, uint32_t tn, uint32_t tm,
    uint32_t splits, i32x4* sums, typename Elem<kType>::T* out, int64_t out_stride) {
    typedef Tile<kType, FN, FM, WN, WM> S;
    typedef typename Elem<kType>::T T;
    extern __shared__ __attribute__((aligned(16))) int8_t lds[];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int wn = wave % WN, wm = wave / WN;
    const int row_stages = ld / kStage;
    const uint32_t total = tn * tm * (kSplit ? splits : 1);
    // a tile's first stage of its row, and its stages
    auto stages_of = [&](uint32_t t, int& from) {
        if (!kSplit) {
            from = 0;
            return row_stages;
        }
        const uint32_t q = t % splits;
        from = (int)(row_stages * q / splits);
        return (int)(row_stages * (q + 1) / splits) - from;
    };

    // What is loaded next: a stage of a tile (behind the last tile its last
    // stage again).  This thread's words: row r0 + i * kRowsPerLoad, word tid % 8.
    const int r0 = tid / 8, c0 = tid % 8;
    const int8_t *wbase, *xbase;
    uint32_t off[S::kLoads];
    uint32_t ftile = blockIdx.x;
    int fstage = 0, fstages;
    auto aim = [&](uint32_t t) {
        uint32_t in, im;
        tile_of(kSplit ? t / splits : t, tn, tm, in, im);
        const int64_t n0 = (int64_t)in * S::BN, m0 = (int64_t)im * S::BM;
        int from;
        fstages = stages_of(t, from);
        wbase = b + n0 * ld + from * kStage;
        xbase = a + m0 * ld + from * kStage;
        const int nlast = (int)(n - n0 < S::BN ? n - n0 : S::BN) - 1;
        const int mlast = (int)(m - m0 < S::BM ? m - m0 : S::BM) - 1;
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) {
            const int r = r0 + i * S::kRowsPerLoad;
            // rows past the end read the last row; their products are not stored
            const int g = r < S::BN ? min(r, nlast) : min(r - S::BN, mlast);
            off[i] = (uint32_t)g * (uint32_t)ld + c0 * 16;
        }
    };
    auto advance = [&]() {
        if (++fstage < fstages) return;
        if (ftile + gridDim.x < total) {
            ftile += gridDim.x;
            fstage = 0;
            aim(ftile);
        } else {
            fstage = fstages - 1;
        }
    };
    const int wslot = r0 * kStage + ((c0 ^ (r0 / 2 & 7)) * 16);
    constexpr int kHalf = S::kLoads / 2;
    i32x4 g[S::kLoads];
    auto fetch = [&](int from, int to) {
        const int64_t k = (int64_t)fstage * kStage;
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) {
            if (i < from || i >= to) continue;
            const int8_t* p = (i * S::kRowsPerLoad < S::BN ? wbase : xbase) + k;
            g[i] = *(const i32x4*)(p + off[i]);
        }
    };
    auto put = [&](int half, int from, int to) {
        int8_t* d = lds + half * S::kStageBytes + wslot;
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i)
            if (i >= from && i < to) *(i32x4*)(d + i * S::kRowsPerLoad * kStage) = g[i];
    };
    i32x4 fa[2][FN], fb[2][FM];
    const int ra = (wn * FN * 32 + (lane & 31)) * kStage;
    const int rb = (S::BN + wm * FM * 32 + (lane & 31)) * kStage;
    int slot[4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) slot[ks] = ((ks * 2 + (lane >> 5)) ^ (lane / 2 & 7)) * 16;
    auto read = [&](int p, int half, int ks) {
        const int8_t* d = lds + half * S::kStageBytes + slot[ks];
#pragma unroll
        for (int f = 0; f < FN; ++f) fa[p][f] = *(const i32x4*)(d + ra + f * 32 * kStage);
#pragma unroll
        for (int f = 0; f < FM; ++f) fb[p][f] = *(const i32x4*)(d + rb + f * 32 * kStage);
    };
    i32x16 acc[FN][FM];
    auto products = [&](int p) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[p][i], fb[p][j], acc[i][j], 0, 0, 0);
    };
    // a step's order: its products with the LDS reads, then the writes, then the
    // loads between them
    constexpr int kReads = FN + FM, kProducts = FN * FM;
#define TILE_STEP(writes, loads)                                                     \
    do {                                                                             \
        constexpr int kFirst = kProducts / 4;                                        \
        _Pragma("unroll") for (int q = 0; q < kFirst; ++q) {                         \
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                       \
            __builtin_amdgcn_sched_group_barrier(0x100, kReads / kFirst, 0);         \
        }                                                                            \
        _Pragma("unroll") for (int q = 0; q < kProducts - kFirst; ++q) {             \
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                       \
            if ((writes) && q < kHalf) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0); \
            if ((loads) && q < kHalf) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0); \
        }                                                                            \
        __builtin_amdgcn_sched_barrier(0);                                           \
    } while (0)
    // A tile's scales and bias lie in LDS (two places by turns); they are loaded
    // a tile ahead.
    float* places = (float*)(lds + 2 * S::kStageBytes);
    float scales[S::kScalesEach];
    auto load_scales = [&](uint32_t t) {
        uint32_t in, im;
        tile_of(t, tn, tm, in, im);
        const int64_t n0 = (int64_t)in * S::BN, m0 = (int64_t)im * S::BM;
#pragma unroll
        for (int i = 0; i < S::kScalesEach; ++i) {
            const int q = i * S::kThreads + tid;
            float v = 0.0f;
            if (q < S::BN) { if (n0 + q < n) v = b_scale[n0 + q]; }
            else if (q < 2 * S::BN) { if (bias && n0 + q - S::BN < n) v = Elem<kType>::up(bias[n0 + q - S::BN]); }
            else if (q < S::kScales) { if (m0 + q - 2 * S::BN < m) v = a_scale[m0 + q - 2 * S::BN]; }
            scales[i] = v;
        }
    };
    auto put_scales = [&](int place) {
#pragma unroll
        for (int i = 0; i < S::kScalesEach; ++i) places[place * S::kPlace + i * S::kThreads + tid] = scales[i];
    };
    if (!kSplit) load_scales(blockIdx.x);
    aim(ftile);
    fetch(0, S::kLoads);
    advance();
    if (!kSplit) put_scales(0);
    put(0, 0, S::kLoads);
    fetch(0, S::kLoads);
    advance();
    __syncthreads();
    read(0, 0, 0);
    int half = 0, turn = 0;
    for (uint32_t t = blockIdx.x; t < total; t += gridDim.x) {
        uint32_t in, im;
        tile_of(kSplit ? t / splits : t, tn, tm, in, im);
        const int64_t n0 = (int64_t)in * S::BN, m0 = (int64_t)im * S::BM;
        if (!kSplit) load_scales(t + gridDim.x < total ? t + gridDim.x : t);
        int from;
        const int stages = stages_of(t, from);
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
        __builtin_amdgcn_sched_barrier(0);
        for (int s = 0; s < stages; ++s) {
            read(1, half, 1);
            products(0);
            put(half ^ 1, 0, kHalf);
            TILE_STEP(true, false);
            read(0, half, 2);
            products(1);
            put(half ^ 1, kHalf, S::kLoads);
            fetch(0, kHalf);
            TILE_STEP(true, true);
            read(1, half, 3);
            products(0);
            fetch(kHalf, S::kLoads);
            TILE_STEP(false, true);
            advance();
            __syncthreads();
            read(0, half ^ 1, 0);
            products(1);
            TILE_STEP(false, false);
            half ^= 1;
        }

        if constexpr (kSplit) {
            i32x4* d = sums + (int64_t)t * (FN * FM * 4 * S::kThreads) + tid;
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        d[((i * FM + j) * 4 + q) * S::kThreads] =
                            i32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
            __builtin_amdgcn_sched_barrier(0);
            continue;
        }
        // Out through the stage's half of LDS that has just been read for the last
        // time, a strip of kStrip tokens x FN * 32 channels of a wave at a time,
        // so that whole lines are stored.  The loads under way are waited for
        // first: later it would be for the stores as well.
        __builtin_amdgcn_s_waitcnt(0x0F70);      // vmcnt(0)
        put_scales(turn ^ 1);
        const float* place = places + turn * S::kPlace;
        turn ^= 1;
        constexpr int kRowBytes = FN * 32 * (int)sizeof(T) + 16;
        constexpr int kSpace = S::kStageBytes / (WN * WM), kStrip = kSpace >= 32 * kRowBytes ? 32 : 16;
        static_assert(kStrip * kRowBytes <= kSpace, "strips fit");
        int8_t* strip = lds + (half ^ 1) * S::kStageBytes + wave * kSpace;
        const int64_t nw = n0 + wn * FN * 32;
        const float *ws = place + wn * FN * 32, *bs = ws + S::BN, *as = place + 2 * S::BN + wm * FM * 32;
        constexpr int kWords = FN * 32 * (int)sizeof(T) / 16;    // 16-byte words of a strip's row
        constexpr int E = Elem<kType>::kE;
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            const int64_t mf = m0 + (wm * FM + f) * 32;
            const float s = as[f * 32 + (lane & 31)];
#pragma unroll
            for (int part = 0; part < 32; part += kStrip) {
                if (kStrip == 32 || (lane & 31) / kStrip == part / kStrip)
#pragma unroll
                    for (int c = 0; c < FN; ++c)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int j = c * 32 + 8 * q + 4 * (lane >> 5);
                            float y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                y[e] = (float)acc[c][f][4 * q + e] * (s * ws[j + e]) + bs[j + e];
                            int8_t* d = strip + ((lane & 31) - part) * kRowBytes + j * (int)sizeof(T);
                            if (kType == FLASHOPT_FP32)
                                *(u32x4*)d = u32x4{as_u32(y[0]), as_u32(y[1]), as_u32(y[2]), as_u32(y[3])};
                            else
                                *(u32x2*)d = pack4<kType>(y);
                        }
                // the strip is this wave's own: its writes come before its reads
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int q = 0; q < kStrip * kWords / kWave; ++q) {
                    const int at = q * kWave + lane, row = at / kWords, word = at % kWords;
                    const u32x4 v = *(const u32x4*)(strip + row * kRowBytes + word * 16);
                    const int64_t i = mf + part + row, j = nw + word * E;
                    if (i < m && j + E <= n) __builtin_nontemporal_store(v, (u32x4_any*)(out + i * out_stride + j));
                    else if (i < m && j < n) store_vec<kType>(out + i * out_stride + nw, word, n - nw, v);
                }
                __builtin_amdgcn_wave_barrier();
            }
        }
        __syncthreads();                         // the strips make way for a stage
        __builtin_amdgcn_sched_barrier(0);
    }
#undef TILE_STEP
}

// The pieces of a tile added up: one block for one of its FN * FM fragments.
template <int kType, int FN, int FM, int WN, int WM>
__global__ __launch_bounds__(WN * WM * kWave) void join_kernel(
    const i32x4* sums, uint32_t splits, const float* a_scale, const float* b_scale,
    const typename Elem<kType>::T* bias, int64_t m, int64_t n, uint32_t tn, uint32_t tm,
    typename Elem<kType>::T* out, int64_t out_stride) {
    typedef Tile<kType, FN, FM, WN, WM> S;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const uint32_t t = blockIdx.x / (FN * FM), f = blockIdx.x % (FN * FM);
    uint32_t in, im;
    tile_of(t, tn, tm, in, im);
    const int64_t i = (int64_t)im * S::BM + (wave / WN * FM + f % FM) * 32 + (lane & 31);
    const int64_t j0 = (int64_t)in * S::BN + (wave % WN * FN + f / FM) * 32 + 4 * (lane >> 5);
    constexpr int64_t kPiece = FN * FM * 4 * S::kThreads;
    const i32x4* p = sums + (int64_t)t * splits * kPiece + f * 4 * S::kThreads + tid;
    i32x4 v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = p[q * S::kThreads];
    for (uint32_t k = 1; k < splits; ++k) {
        p += kPiece;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += p[q * S::kThreads];
    }
    if (i >= m) return;
    const float s = a_scale[i];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t j = j0 + 8 * q + e;
            if (j >= n) continue;
            float y = (float)v[q][e] * (s * b_scale[j]);
            if (bias) y += Elem<kType>::up(bias[j]);
            out[i * out_stride + j] = Elem<kType>::down(y);
        }
}

// ---- the product: few tokens ------------------------------------------------------

// Up to 16 MT tokens: the weights are read once, straight into registers, at
// the rate of HBM, and the tokens come from the caches.  A block takes 16
// output channels, its 8 waves a share of the row each (v_mfma_i32_16x16x64_i8:
// lane l holds 16 codes of channel or token l % 16), and adds their integer
// sums up in LDS.
constexpr int kSkinnyWaves = 8;

// What a block's waves leave: their sums of 16 channels x 16 MT tokens.
template <int MT, int kWaves>
struct SkinnySums {
    int v[kWaves][MT][16][17];
};

// A block's output.  A thread's entries are of channel n0 + threadIdx.x % 16, whose
// scale and bias are loaded before the weights, as loads come back in order
// (behind them: 14.5 us for 12.5 at 16 tokens, 50257 x 768), and so are its
// tokens' scales, where they do not come from LDS.
template <int kType, int MT, int kWaves>
struct SkinnyOut {
    static constexpr int kRows = kWaves * 4, kEach = (MT * 16 + kRows - 1) / kRows;
    float channel, bias, token[kEach];
    int m;
    int64_t n0, n;

    __device__ __forceinline__ SkinnyOut(const float* a_scale, const float* b_scale,
                                         const typename Elem<kType>::T* b, int m_, int64_t n0_,
                                         int64_t n_)
        : m(m_), n0(n0_), n(n_) {
        const int64_t j = min(n0 + (threadIdx.x & 15), n - 1);
        channel = b_scale[j];
        bias = b ? Elem<kType>::up(b[j]) : 0.0f;
        if (a_scale)
#pragma unroll
            for (int r = 0; r < kEach; ++r) token[r] = a_scale[min(r * kRows + (int)threadIdx.x / 16, m - 1)];
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ void write(SkinnySums<MT, kWaves>& sums, const i32x4* acc,
                                          typename Elem<kType>::T* out, int64_t out_stride,
                                          const float* scale = nullptr) const {
        const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) sums.v[wave][t][lane & 15][(lane >> 4) * 4 + r] = acc[t][r];
        __syncthreads();
        const int j = threadIdx.x & 15;
#pragma unroll
        for (int r = 0; r < kEach; ++r) {
            const int i = r * kRows + threadIdx.x / 16;
            if (i >= m || i >= MT * 16 || n0 + j >= n) continue;
            int sum = 0;
#pragma unroll
            for (int v = 0; v < kWaves; ++v) sum += sums.v[v][i / 16][i % 16][j];
            out[(int64_t)i * out_stride + n0 + j] =
                Elem<kType>::down((float)sum * ((scale ? scale[i] : token[r]) * channel) + bias);
        }
    }
};

// A wave's share of a row, in lines of 128 codes.
template <int kWaves>
struct SkinnyShare {
    int k, end;
    __device__ __forceinline__ SkinnyShare(int32_t ld, int wave) {
        const int lines = ld / 128;
        k = lines * wave / kWaves * 128;
        end = lines * (wave + 1) / kWaves * 128;
    }
};
constexpr int kSkinnyWords = 8;                  // of 64 codes, in flight at a time

template <int kType, int MT>
__global__ __launch_bounds__(kSkinnyWaves * kWave) void skinny_kernel(
    const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale,
    const typename Elem<kType>::T* bias, int m, int64_t n, int32_t ld,
    typename Elem<kType>::T* out, int64_t out_stride) {
    __shared__ SkinnySums<MT, kSkinnyWaves> sums;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const SkinnyOut<kType, MT, kSkinnyWaves> to(a_scale, b_scale, bias, m, n0, n);
    const int8_t* w = b + min(n0 + (lane & 15), n - 1) * ld + (lane >> 4) * 16;
    const int8_t* x[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) x[t] = a + (int64_t)min(t * 16 + (lane & 15), m - 1) * ld + (lane >> 4) * 16;
    i32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = i32x4{0, 0, 0, 0};
    SkinnyShare<kSkinnyWaves> s(ld, wave);
    auto some = [&](auto count) {
        constexpr int L = decltype(count)::value;
        i32x4 wv[L];
#pragma unroll
        for (int i = 0; i < L; ++i) wv[i] = *(const i32x4*)(w + s.k + i * 64);
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
            for (int t = 0; t < MT; ++t)
                acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[i], *(const i32x4*)(x[t] + s.k + i * 64), acc[t], 0, 0, 0);
        s.k += L * 64;
    };
    while (s.k + kSkinnyWords * 64 <= s.end) some(std::integral_constant<int, kSkinnyWords>());
    while (s.k < s.end) some(std::integral_constant<int, 2>());
    to.write(sums, acc, out, out_stride);
}

// The same for up to kFewTokens tokens in their own type, which each block
// rounds for itself into LDS while its first weights are on their way: one
// launch, no workspace.
constexpr int kFewTokens = 4, kFewEntries = 16;  // entries of a token that a thread holds

template <int kType, int kWaves>
__global__ __launch_bounds__(kWaves * kWave) void few_kernel(
    const typename Elem<kType>::T* x, int m, int32_t cols, int64_t x_stride, const int8_t* b,
    const float* b_scale, const typename Elem<kType>::T* bias, int64_t n, int32_t ld,
    typename Elem<kType>::T* out, int64_t out_stride) {
    constexpr int E = Elem<kType>::kE;
    extern __shared__ __attribute__((aligned(16))) int8_t codes[];       // m rows of ld + 16
    __shared__ SkinnySums<1, kWaves> sums;
    __shared__ uint32_t red[kWaves];
    __shared__ float scale[kFewTokens];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    // the waves of a row; its words and the entries behind them
    const int each = kWaves / (m <= 1 ? 1 : m <= 2 ? 2 : 4), row = wave / each, at = wave % each * kWave + lane;
    const int step = each * kWave, words = cols / E, left = cols % E;
    const typename Elem<kType>::T* p = x + (int64_t)min(row, m - 1) * x_stride;
    // The tokens' loads go first and without a branch: loads come back in order, so
    // that their largest entry is found while the weights are still on their way.
    // Words past the row's end read its last word again.
    constexpr int kHeld = kFewEntries / E;
    u32x4 xv[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        xv[i] = *reinterpret_cast<const u32x4_any*>(p + min(i * step + at, words - 1) * E);
    const float rest = Elem<kType>::up(p[at < left ? words * E + at : 0]);
    const SkinnyOut<kType, 1, kWaves> to(nullptr, b_scale, bias, m, n0, n);

    const int8_t* w = b + min(n0 + (lane & 15), n - 1) * ld + (lane >> 4) * 16;
    SkinnyShare<kWaves> s(ld, wave);
    i32x4 wv[kSkinnyWords];
    const int first = s.end - s.k < kSkinnyWords * 64 ? s.end - s.k : kSkinnyWords * 64;
    // words past the share are read from its row and not used (ld is at least 128)
#pragma unroll
    for (int i = 0; i < kSkinnyWords; ++i) wv[i] = *(const i32x4*)(w + (i * 64 < first ? s.k + i * 64 : 0));
    __builtin_amdgcn_sched_barrier(0);

    uint32_t top = as_u32(rest) & 0x7FFFFFFFu;   // (or of the row's first entry)
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) top = max(top, as_u32(Elem<kType>::get(xv[i], e)) & 0x7FFFFFFFu);
    top = wave_max_u32(top);
    if (lane == 0) red[wave] = top;
    __syncthreads();
    for (int q = 0; q < each; ++q) top = max(top, red[row * each + q]);
    const RowScale S(top);
    if (row < m) {
        int8_t* q = codes + row * (ld + 16);
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (i * step + at < words) word_codes<kType>(xv[i], (i * step + at) * E, cols, S, q);
        if (at < left) q[words * E + at] = (int8_t)S.code(rest);
        for (int j = cols + at; j < ld; j += step) q[j] = 0;
        if (at == 0) scale[row] = S.scale();
    }
    __syncthreads();
    const int8_t* xl = codes + min(lane & 15, m - 1) * (ld + 16) + (lane >> 4) * 16;
    i32x4 acc = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kSkinnyWords; ++i)
        if (i * 64 < first)
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[i], *(const i32x4*)(xl + s.k + i * 64), acc, 0, 0, 0);
    s.k += first;
    auto some = [&](auto count) {
        constexpr int L = decltype(count)::value;
#pragma unroll
        for (int i = 0; i < L; ++i) wv[i] = *(const i32x4*)(w + s.k + i * 64);
#pragma unroll
        for (int i = 0; i < L; ++i)
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[i], *(const i32x4*)(xl + s.k + i * 64), acc, 0, 0, 0);
        s.k += L * 64;
    };
    while (s.k + kSkinnyWords * 64 <= s.end) some(std::integral_constant<int, kSkinnyWords>());
    while (s.k < s.end) some(std::integral_constant<int, 2>());
    to.write(sums, &acc, out, out_stride, scale);
}

template <typename F>
static int by_type(int32_t type, F f) {
    if (type == FLASHOPT_BF16) f(std::integral_constant<int, FLASHOPT_BF16>());
    else if (type == FLASHOPT_FP16) f(std::integral_constant<int, FLASHOPT_FP16>());
    else f(std::integral_constant<int, FLASHOPT_FP32>());
    return launch_status();
}

static constexpr int64_t kMaxRows = int64_t(1) << 24;

static int check_matrix(int64_t rows, int64_t cols) {
    if (rows < 0 || rows > kMaxRows || cols < 1 || cols > FLASHOPT_INT8_COLS_MAX)
        return FLASHOPT_ERR_SIZE;
    return FLASHOPT_OK;
}

// the product's tiles are counted in 32 bits
static int check_outputs(int64_t m, int64_t n) {
    return (m / 128 + 1) * (n / 128 + 1) > (int64_t(1) << 30) ? FLASHOPT_ERR_SIZE : FLASHOPT_OK;
}

// x is read after the first outputs have been written: every block of
// few_kernel rounds it for itself
static int check_apart(int32_t type, int64_t m, const void* x, int64_t x_stride, int64_t k,
                       const void* out, int64_t out_stride, int64_t n) {
    const int64_t size = (int64_t)type_size(type);
    return overlap(m, x, x_stride * size, k * size, out, out_stride * size, n * size)
               ? FLASHOPT_ERR_ARG : FLASHOPT_OK;
}

static int check_codes(const void* codes, const void* scale) {
    if (!codes || !scale) return FLASHOPT_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scale, 4)) return FLASHOPT_ERR_ALIGN;
    return FLASHOPT_OK;
}

// A launch has less than 2^32 threads: rows in parts of 2^21 blocks.
template <typename F>
static void by_rows(int64_t rows, F f) {
    constexpr int64_t kPart = int64_t(1) << 21;
    for (int64_t first = 0; first < rows; first += kPart)
        f(first, dim3((unsigned)(rows - first < kPart ? rows - first : kPart)));
}

static int launch_quantize(const void* x, int32_t type, int64_t rows, int64_t cols, int64_t stride,
                           int8_t* codes, float* scale, hipStream_t st) {
    const int64_t ld = ld_of(cols);
    return by_type(type, [&](auto k) {
        constexpr int kType = decltype(k)::value, E = Elem<kType>::kE;
        const auto* p = (const typename Elem<kType>::T*)x;
        by_rows(rows, [&](int64_t first, dim3 grid) {
            // the fewest waves and words that hold a row
            if (ld <= 2 * kWave * E)
                hipLaunchKernelGGL((quantize_rows_kernel<kType, 1, 2>), grid, dim3(kWave), 0, st, p,
                                   cols, stride, ld, codes, scale, first);
            else if (ld <= 2 * kBlock * E)
                hipLaunchKernelGGL((quantize_rows_kernel<kType, 4, 2>), grid, dim3(kBlock), 0, st, p,
                                   cols, stride, ld, codes, scale, first);
            else if (ld <= 8 * kBlock * E)
                hipLaunchKernelGGL((quantize_rows_kernel<kType, 16, 2>), grid, dim3(16 * kWave), 0, st,
                                   p, cols, stride, ld, codes, scale, first);
            else
                hipLaunchKernelGGL((quantize_long_kernel<kType>), grid, dim3(kBlock), 0, st, p, cols,
                                   stride, ld, codes, scale, first);
        });
    });
}

template <int kType, int FN, int FM, int WN, int WM>
static void launch_tile(const int8_t* a, const float* a_scale, const int8_t* b,
                        const float* b_scale, const typename Elem<kType>::T* bias, int64_t m,
                        int64_t n, int64_t ld, typename Elem<kType>::T* out, int64_t out_stride,
                        hipStream_t st) {
    typedef Tile<kType, FN, FM, WN, WM> S;
    const int64_t tn = (n + S::BN - 1) / S::BN, tm = (m + S::BM - 1) / S::BM;
    const int64_t most = 256 * S::kBlocks, blocks = tn * tm < most ? tn * tm : most;
    hipLaunchKernelGGL((tile_kernel<kType, FN, FM, WN, WM, false>), dim3((unsigned)blocks),
                       dim3(S::kThreads), S::kLds, st, a, a_scale, b, b_scale, bias, m, n,
                       (int32_t)ld, (uint32_t)tn, (uint32_t)tm, 1u, nullptr, out, out_stride);
}

// How a product is done, and what of a workspace it needs.
struct Plan {
    enum Way { kSkinny, kSplit, kSmall, kLarge } way;
    int skinny;                                  // 16 tokens times this
    int64_t splits;
    size_t sums;                                 // bytes
};
typedef Tile<FLASHOPT_FP32, 2, 2, 2, 2> SmallTile;

static Plan plan_of(int64_t m, int64_t n, int64_t k) {
    Plan p = {Plan::kSkinny, 0, 1, 0};
    const int64_t stages = ld_of(k) / kStage;
    const int64_t tn = (n + SmallTile::BN - 1) / SmallTile::BN, tm = (m + SmallTile::BM - 1) / SmallTile::BM;
    const int64_t tiles = tn * tm, large = ((n + 255) / 256) * ((m + 255) / 256);
    // 4096 x 4096 x 4096 in large tiles: 64 us; 2048 x 4096 x 4096 in small ones 40
    // for 47, 1024 x 5120 x 5120 40 for 63.  Half of a large tile is waste up to 128
    // rows of a side: 64 tokens, 128256 x 4096: 127 us in small ones for 144; 150: 165
    // for 150.
    if (large >= 200 && m > 128 && n > 128) {
        p.way = Plan::kLarge;
        return p;
    }
    // Pieces of at least 8 stages, until a block runs on each CU, if that gains:
    // a stage takes about half a microsecond of a block alone on its CU, another
    // launch 6, a piece's sums 1/32.  100 tokens, 4096 x 14336 (32 tiles): 34 us
    // for 66; 1024 x 4096 (8 tiles): 20 for 24; but 128 tokens, 14336 x 4096 (112
    // tiles): 31 for 22.
    const int64_t q = 256 / tiles < stages / 8 ? 256 / tiles : stages / 8;
    const bool split = q >= 2 && stages * (q - 1) * 16 > q * (192 + tiles * q);
    // Up to 16 tokens the weights' own rate decides.  Up to 64 the tokens read
    // again for every 16 channels count, and tiles need channels to fill the GPU:
    // each way's time in 1/256 us, fitted to 180 sizes of 17 to 64 tokens, 768 to
    // 11264 channels and rows of 768 to 28672.  Within 18% of the better way at
    // each (14.9 us for 12.7 at worst), 0.2% over them all; 64 tokens of 4096 x
    // 4096: 12 us here, 18 in tiles; of 4096 x 14336: 40 and 27.
    const int64_t here = 512 + stages * (m + 26) * (n > 4096 ? n : 4096) / 4096;
    const int64_t in_tiles = split ? 3840 + 205 * stages / q : 1024 + 192 * stages;
    if (m <= 16 || (m <= 64 && tn < 96 && here <= in_tiles)) {
        p.skinny = m <= 16 ? 1 : m <= 32 ? 2 : 4;
        return p;
    }
    p.way = Plan::kSmall;
    if (split) {
        p.way = Plan::kSplit;
        p.splits = q;
        p.sums = (size_t)(tiles * q) * (SmallTile::BN * SmallTile::BM * sizeof(int));
    }
    return p;
}

static int launch_matmul(const Plan& plan, const int8_t* a, const float* a_scale, const int8_t* b,
                         const float* b_scale, const void* bias, int64_t m, int64_t n, int64_t k,
                         void* out, int32_t type, int64_t out_stride, void* sums, hipStream_t st) {
    return by_type(type, [&](auto t) {
        constexpr int kType = decltype(t)::value;
        typedef typename Elem<kType>::T T;
        const int64_t ld = ld_of(k);
        const T* bi = (const T*)bias;
        T* o = (T*)out;
        auto skinny = [&](auto mt) {
            constexpr int MT = decltype(mt)::value;
            hipLaunchKernelGGL((skinny_kernel<kType, MT>), dim3((unsigned)((n + 15) / 16)),
                               dim3(kSkinnyWaves * kWave), 0, st, a, a_scale, b, b_scale, bi, (int)m,
                               n, (int32_t)ld, o, out_stride);
        };
        if (plan.way == Plan::kLarge) {
            launch_tile<kType, 2, 4, 4, 2>(a, a_scale, b, b_scale, bi, m, n, ld, o, out_stride, st);
        } else if (plan.way == Plan::kSmall) {
            launch_tile<kType, 2, 2, 2, 2>(a, a_scale, b, b_scale, bi, m, n, ld, o, out_stride, st);
        } else if (plan.way == Plan::kSplit) {
            typedef SmallTile S;
            const uint32_t tn = (uint32_t)((n + S::BN - 1) / S::BN), tm = (uint32_t)((m + S::BM - 1) / S::BM);
            hipLaunchKernelGGL((tile_kernel<FLASHOPT_FP32, 2, 2, 2, 2, true>),
                               dim3((unsigned)(tn * tm * plan.splits)), dim3(S::kThreads), S::kLds, st,
                               a, a_scale, b, b_scale, nullptr, m, n, (int32_t)ld, tn, tm,
                               (uint32_t)plan.splits, (i32x4*)sums, nullptr, 0);
            hipLaunchKernelGGL((join_kernel<kType, 2, 2, 2, 2>), dim3(tn * tm * 4), dim3(S::kThreads),
                               0, st, (const i32x4*)sums, (uint32_t)plan.splits, a_scale, b_scale, bi,
                               m, n, tn, tm, o, out_stride);
        } else if (plan.skinny == 1) {
            skinny(std::integral_constant<int, 1>());
        } else if (plan.skinny == 2) {
            skinny(std::integral_constant<int, 2>());
        } else {
            skinny(std::integral_constant<int, 4>());
        }
    });
}

// Rounding the tokens in every block saves a launch and pays while the threads
// hold the tokens and either the blocks all run at once or the rows are long:
// the waves of a block, 0 for two launches.  Measured over weights that are read
// again and again, the GPU's time here and in two launches: 1 token: 4096 x 4096
// 5.3 and 8.2 us, 14336 x 4096 11.5 and 15.9 (12 weights by turns, which no cache
// holds: 14.2 and 17.4), 128256 x 4096 87 and 90, 28672 x 8192 40.1 and 40.2, but 50257
// x 768 (3142 blocks) 17.2 and 12.4 (of 2048: 18.4 and 21.0); 2 tokens, 4096 x 4096:
// 6.8 and 8.9; 4 tokens, 4096 x 2048: 5.6 and 6.6, 2304 x 768: 5.1 and 6.4.  Blocks of 4
// waves leave room for more of them: 1 token, 14336 x 4096: 11.5 us, 14.0 with 8
// waves; up to one block a CU 8 waves read faster (4096 x 4096: 5.3 for 6.7).
static int few_waves(int64_t m, int64_t n, int64_t k) {
    const int64_t blocks = (n + 15) / 16, rows = m <= 1 ? 1 : m <= 2 ? 2 : 4;
    if (m > kFewTokens || k < 8 || (blocks > 1024 && k < 4096)) return 0;
    const int64_t held = kFewEntries * kWave / rows;             // of a token, by each wave
    if (blocks > 256 && k <= 4 * held) return 4;
    return k <= 8 * held ? 8 : 0;
}

static size_t up256(size_t b) { return (b + 255) & ~size_t(255); }

}  // namespace flashopt

using namespace flashopt;

extern "C" {

int64_t flashopt_int8_ld(int64_t cols) {
    return cols < 1 || cols > FLASHOPT_INT8_COLS_MAX ? 0 : ld_of(cols);
}

int flashopt_quantize_rows(const void* x, int32_t type, int64_t rows, int64_t cols,
                           int64_t stride, int8_t* codes, float* scale, void* stream) {
    if (!valid_type(type)) return FLASHOPT_ERR_ARG;
    const int e = check_matrix(rows, cols);
    if (e) return e;
    if (stride < cols || stride > kMaxNumel) return FLASHOPT_ERR_SIZE;
    if (rows == 0) return FLASHOPT_OK;
    if (!x) return FLASHOPT_ERR_NULL;
    if (!aligned(x, type_size(type))) return FLASHOPT_ERR_ALIGN;
    const int c = check_codes(codes, scale);
    if (c) return c;
    return launch_quantize(x, type, rows, cols, stride, codes, scale, (hipStream_t)stream);
}

int flashopt_tensor_quantize_rows(const flashopt_tensor* t, int32_t kind, int64_t cols,
                                  int8_t* codes, float* scale, void* stream) {
    if (!t) return FLASHOPT_ERR_NULL;
    if (!valid_kind(kind)) return FLASHOPT_ERR_ARG;
    const int s = check_tensor(*t, kind);
    if (s) return s;
    if (cols < 1 || t->numel % cols != 0) return FLASHOPT_ERR_SIZE;
    const int64_t rows = t->numel / cols;
    const int e = check_matrix(rows, cols);
    if (e) return e;
    if (rows == 0) return FLASHOPT_OK;
    const int c = check_codes(codes, scale);
    if (c) return c;
    const DevTensor d = to_dev(*t);
    const int64_t ld = ld_of(cols);
    hipStream_t st = (hipStream_t)stream;
    const bool adam = opt_of(kind) == kAdamW, fp32 = is_fp32(kind);      // SGD and Lion share a layout
    by_rows(rows, [&](int64_t first, dim3 grid) {
        auto launch = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, grid, dim3(kBlock), 0, st, d, cols, ld, codes, scale, first);
        };
        if (fp32 && adam) launch(quantize_state_kernel<kAdamW, true>);
        else if (fp32) launch(quantize_state_kernel<kSgd, true>);
        else if (adam) launch(quantize_state_kernel<kAdamW, false>);
        else launch(quantize_state_kernel<kSgd, false>);
    });
    return launch_status();
}

size_t flashopt_int8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (check_matrix(m, k) || check_matrix(n, k) || check_outputs(m, n) || m == 0 || n == 0 || few_waves(m, n, k)) return 0;
    return up256(plan_of(m, n, k).sums) + up256((size_t)(m * ld_of(k))) +
           up256((size_t)m * sizeof(float));
}

size_t flashopt_int8_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (check_matrix(m, k) || check_matrix(n, k) || check_outputs(m, n) || m == 0 || n == 0) return 0;
    return plan_of(m, n, k).sums;
}

static int check_product(const int8_t* a, const float* a_scale, const int8_t* b,
                         const float* b_scale, const void* bias, const void* out, int32_t type) {
    const int c = check_codes(a, a_scale);
    if (c) return c;
    const int w = check_codes(b, b_scale);
    if (w) return w;
    if (!out) return FLASHOPT_ERR_NULL;
    if (!aligned(out, type_size(type)) || !aligned(bias, type_size(type))) return FLASHOPT_ERR_ALIGN;
    return FLASHOPT_OK;
}

int flashopt_int8_matmul(const int8_t* a, const float* a_scale, const int8_t* b,
                         const float* b_scale, const void* bias, int64_t m, int64_t n, int64_t k,
                         void* out, int32_t out_type, int64_t out_stride, void* workspace,
                         size_t workspace_bytes, void* stream) {
    if (!valid_type(out_type)) return FLASHOPT_ERR_ARG;
    if (check_matrix(m, k) || check_matrix(n, k) || check_outputs(m, n) || out_stride < n || out_stride > kMaxNumel)
        return FLASHOPT_ERR_SIZE;
    if (m == 0 || n == 0) return FLASHOPT_OK;
    const int e = check_product(a, a_scale, b, b_scale, bias, out, out_type);
    if (e) return e;
    const Plan plan = plan_of(m, n, k);
    if (plan.sums) {
        if (!workspace) return FLASHOPT_ERR_NULL;
        if (workspace_bytes < plan.sums || !aligned(workspace, 256)) return FLASHOPT_ERR_WORKSPACE;
    }
    return launch_matmul(plan, a, a_scale, b, b_scale, bias, m, n, k, out, out_type, out_stride,
                         workspace, (hipStream_t)stream);
}

int flashopt_int8_linear(const void* x, int32_t type, int64_t m, int64_t k, int64_t x_stride,
                         const int8_t* w, const float* w_scale, const void* bias, int64_t n,
                         void* out, int64_t out_stride, void* workspace, size_t workspace_bytes,
                         void* stream) {
    if (!valid_type(type)) return FLASHOPT_ERR_ARG;
    if (check_matrix(m, k) || check_matrix(n, k) || check_outputs(m, n) || out_stride < n || out_stride > kMaxNumel ||
        x_stride < k || x_stride > kMaxNumel)
        return FLASHOPT_ERR_SIZE;
    if (m == 0 || n == 0) return FLASHOPT_OK;
    if (!x) return FLASHOPT_ERR_NULL;
    if (!aligned(x, type_size(type))) return FLASHOPT_ERR_ALIGN;
    hipStream_t st = (hipStream_t)stream;
    const int few = few_waves(m, n, k);
    if (few) {
        const int e = check_product(w, w_scale, w, w_scale, bias, out, type);
        if (e) return e;
        if (check_apart(type, m, x, x_stride, k, out, out_stride, n)) return FLASHOPT_ERR_ARG;
        return by_type(type, [&](auto t) {
            constexpr int kType = decltype(t)::value;
            typedef typename Elem<kType>::T T;
            const int64_t ld = ld_of(k);
            auto launch = [&](auto waves) {
                constexpr int kWaves = decltype(waves)::value;
                hipLaunchKernelGGL((few_kernel<kType, kWaves>), dim3((unsigned)((n + 15) / 16)),
                                   dim3(kWaves * kWave), (size_t)(m * (ld + 16)), st, (const T*)x,
                                   (int)m, (int32_t)k, x_stride, w, w_scale, (const T*)bias, n,
                                   (int32_t)ld, (T*)out, out_stride);
            };
            if (few == 4) launch(std::integral_constant<int, 4>());
            else launch(std::integral_constant<int, 8>());
        });
    }
    if (!workspace) return FLASHOPT_ERR_NULL;
    if (workspace_bytes < flashopt_int8_workspace_bytes(m, n, k) || !aligned(workspace, 256))
        return FLASHOPT_ERR_WORKSPACE;
    const Plan plan = plan_of(m, n, k);
    int8_t* codes = (int8_t*)workspace + up256(plan.sums);
    float* scale = (float*)(codes + up256((size_t)(m * ld_of(k))));
    const int e = check_product(codes, scale, w, w_scale, bias, out, type);
    if (e) return e;
    if (check_apart(type, m, x, x_stride, k, out, out_stride, n)) return FLASHOPT_ERR_ARG;
    const int q = launch_quantize(x, type, m, k, x_stride, codes, scale, st);
    if (q) return q;
    return launch_matmul(plan, codes, scale, w, w_scale, bias, m, n, k, out, type, out_stride,
                         workspace, st);
}

}  // extern "C"
