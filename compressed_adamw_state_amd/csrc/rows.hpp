// Element types and wave helpers of the language-model operators
// (include/flashopt_lm.h): 16-byte accesses of BF16, FP16 and FP32 rows that
// start at any element, reductions over a wave, and the host's checks.
#pragma once

#include "host.hpp"
#include "flashopt_lm.h"

namespace flashopt {

// Rows of an odd length start at any multiple of the element size, so their
// 16-byte accesses are declared with that alignment only.  gfx950 serves them
// as one access; one that straddles a line costs one more line.
typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <int kType> struct Elem;                // kE elements in 16 bytes
template <> struct Elem<FLASHOPT_BF16> {
    typedef uint16_t T;
    static constexpr int kE = 8;
    static __device__ __forceinline__ float get(const u32x4& v, int e) {
        const uint32_t w = v[e >> 1];
        return as_f32((e & 1) ? (w & 0xFFFF0000u) : (w << 16));
    }
    static __device__ __forceinline__ float up(T b) { return as_f32((uint32_t)b << 16); }
    static __device__ __forceinline__ T down(float x) {
        return __builtin_bit_cast(uint16_t, (__bf16)x);
    }
    static constexpr uint32_t kMinusInf = 0xFF80FF80u;
};
template <> struct Elem<FLASHOPT_FP16> {
    typedef uint16_t T;
    static constexpr int kE = 8;
    static __device__ __forceinline__ float get(const u32x4& v, int e) {
        const uint32_t w = v[e >> 1];
        return (float)__builtin_bit_cast(_Float16, (uint16_t)((e & 1) ? w >> 16 : w));
    }
    static __device__ __forceinline__ float up(T b) { return f16_to_f32(b); }
    static __device__ __forceinline__ T down(float x) { return (T)f32_to_f16(x); }
    static constexpr uint32_t kMinusInf = 0xFC00FC00u;
};
template <> struct Elem<FLASHOPT_FP32> {
    typedef uint32_t T;
    static constexpr int kE = 4;
    static __device__ __forceinline__ float get(const u32x4& v, int e) { return as_f32(v[e]); }
    static __device__ __forceinline__ float up(T b) { return as_f32(b); }
    static __device__ __forceinline__ T down(float x) { return as_u32(x); }
    static constexpr uint32_t kMinusInf = 0xFF800000u;
};

// kE values rounded to the type, as one 16-byte word
template <int kType>
__device__ __forceinline__ u32x4 pack(const float* x) {
    u32x4 v;
    if (kType == FLASHOPT_FP32) {
        v = u32x4{as_u32(x[0]), as_u32(x[1]), as_u32(x[2]), as_u32(x[3])};
    } else if (kType == FLASHOPT_BF16) {
        typedef float f2 __attribute__((ext_vector_type(2)));
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{x[2 * i], x[2 * i + 1]}), b2));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = f32_to_f16(x[2 * i]) | (f32_to_f16(x[2 * i + 1]) << 16);
    }
    return v;
}

// Vector v of a row of n elements; entries past the row's end read as `fill`.
template <int kType>
__device__ __forceinline__ u32x4 load_vec(const typename Elem<kType>::T* row, int64_t v, int64_t n,
                                          uint32_t fill) {
    constexpr int E = Elem<kType>::kE;
    const int64_t j = v * E;
    if (j + E <= n) return *reinterpret_cast<const u32x4_any*>(row + j);
    u32x4 r = {fill, fill, fill, fill};
    if (j < n) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (j + e < n) {
                if (kType == FLASHOPT_FP32) {
                    r[e & 3] = row[j + e];
                } else {
                    const uint32_t b = row[j + e];
                    r[e >> 1] = (e & 1) ? ((r[e >> 1] & 0xFFFFu) | (b << 16))
                                        : ((r[e >> 1] & 0xFFFF0000u) | b);
                }
            }
        }
    }
    return r;
}

template <int kType>
__device__ __forceinline__ void store_vec(typename Elem<kType>::T* row, int64_t v, int64_t n,
                                          u32x4 x) {
    constexpr int E = Elem<kType>::kE;
    const int64_t j = v * E;
    if (j + E <= n) {
        *reinterpret_cast<u32x4_any*>(row + j) = x;
    } else if (j < n) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (j + e < n)
                row[j + e] = kType == FLASHOPT_FP32
                                 ? (typename Elem<kType>::T)x[e & 3]
                                 : (typename Elem<kType>::T)((e & 1) ? x[e >> 1] >> 16 : x[e >> 1]);
    }
}

// Reductions over a wave by data-parallel moves: within rows of 16 lanes (shift
// right by 1, 2, 4, 8), then each odd row takes its lower neighbour's last lane and
// the upper half lane 31's, so that lane 63 has all.  About 8 cycles a move,
// where a shuffle through LDS takes about 100.
template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t lane_move(uint32_t none, uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)x, kCtrl, kRows, 0xF, false);
}
template <typename F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t x, uint32_t none, F f) {
    x = f(x, lane_move<0x111, 0xF>(none, x));
    x = f(x, lane_move<0x112, 0xF>(none, x));
    x = f(x, lane_move<0x114, 0xF>(none, x));
    x = f(x, lane_move<0x118, 0xF>(none, x));
    x = f(x, lane_move<0x142, 0xA>(none, x));
    x = f(x, lane_move<0x143, 0xC>(none, x));
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}
__device__ __forceinline__ float wave_max(float x) {
    return as_f32(wave_reduce(as_u32(x), 0xFF800000u, [](uint32_t a, uint32_t b) {
        return as_u32(fmaxf(as_f32(a), as_f32(b)));
    }));
}
__device__ __forceinline__ float wave_sum(float x) {
    return as_f32(wave_reduce(as_u32(x), 0u, [](uint32_t a, uint32_t b) {
        return as_u32(as_f32(a) + as_f32(b));
    }));
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t x) {
    return wave_reduce(x, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const uint64_t y = __shfl_xor((unsigned long long)x, o);
        x = y > x ? y : x;
    }
    return x;
}

// hardware exp2 / log2 (about one ulp; results below 2^-126 become 0)
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_hw(float x) { return __builtin_amdgcn_logf(x); }

constexpr float kLn2 = 0x1.62e43p-1f;            // RN(log 2)
constexpr float kLog2e = 0x1.715476p+0f;         // RN(1 / log 2)

static inline bool valid_type(int32_t type) {
    return type >= FLASHOPT_BF16 && type <= FLASHOPT_FP32;
}
static inline size_t type_size(int32_t type) { return type == FLASHOPT_FP32 ? 4 : 2; }

// Whether two matrices of `rows` rows (strides and row lengths in bytes) have a
// byte in common.  Rows that lie between each other's are told apart where the
// strides are equal; overlapping spans of other strides count as shared.
static inline bool overlap(int64_t rows, const void* a, int64_t a_stride, int64_t a_bytes,
                           const void* b, int64_t b_stride, int64_t b_bytes) {
    typedef __int128 Wide;                       // rows * stride may pass 64 bits
    const Wide p = (uintptr_t)a, q = (uintptr_t)b;
    if (p + (Wide)(rows - 1) * a_stride + a_bytes <= q || q + (Wide)(rows - 1) * b_stride + b_bytes <= p)
        return false;
    if (a_stride != b_stride || rows == 1) return true;
    const Wide d = ((q - p) % a_stride + a_stride) % a_stride;
    return d < a_bytes || a_stride - d < b_bytes;
}

}  // namespace flashopt
