// Activations held in 8 bits and the activation functions that hold their own
// inputs (include/flashopt_lm.h); held.hpp has the codec.
//
// Everything here is one pass over memory, a 16-byte word of the input's type at
// a time, four of them on their way per thread, so HBM is the bound: 8192 x 4096 BF16 held
// in 19 us (5.3 TB/s of reads and writes); 8192 x 14336 gated forward and held 181 us (5.3
// TB/s), backward 173 (5.5), where a large copy reaches 4.9.  A word's codes cost 2.75
// instructions a value (product and rounding in one fma, bound, a quarter of three
// permutes), its values back 2 (conversion from a byte, product).
#include <utility>

#include "held.hpp"

namespace flashopt {

constexpr int kHoldWords = 4;                    // a thread's words, all loaded before the first is used
constexpr int64_t kHoldBlocks = int64_t(1) << 22;

template <int kType>
struct HeldOut {                                 // null codes: not held
    int8_t* codes;
    uint8_t* powers;
    // word w of row r: E codes, and the group's byte by its first lane
    __device__ __forceinline__ void put(int64_t ld, int64_t row, uint32_t w, const u32x4& v, bool in) const {
        constexpr int E = Elem<kType>::kE;
        uint32_t c[E / 4];
        const Power p = hold_word<kType>(v, c);
        if (!in) return;
        int8_t* to = codes + row * ld + (int64_t)w * E;
        if (E == 8) *reinterpret_cast<u32x2*>(to) = u32x2{c[0], c[E / 4 - 1]};
        else *reinterpret_cast<uint32_t*>(to) = c[0];
        if (w % (kGroup8 / E) == 0) powers[row * (ld / kGroup8) + w / (kGroup8 / E)] = (uint8_t)p.byte;
    }
};
template <int kType>
struct HeldIn {
    const int8_t* codes;
    const uint8_t* powers;
    struct Word {
        uint32_t c[Elem<kType>::kE / 4], byte;
    };
    __device__ __forceinline__ Word get(int64_t ld, int64_t row, uint32_t w) const {
        constexpr int E = Elem<kType>::kE;
        const int8_t* p = codes + row * ld + (int64_t)w * E;
        Word r;
        if constexpr (E == 8) {
            const u32x2 c = *reinterpret_cast<const u32x2*>(p);
            r.c[0] = c[0];
            r.c[1] = c[1];
        } else {
            r.c[0] = *reinterpret_cast<const uint32_t*>(p);
        }
        r.byte = powers[row * (ld / kGroup8) + w / (kGroup8 / E)];
        return r;
    }
    static __device__ __forceinline__ void values(const Word& w, float* x) {
        const float up = as_f32(w.byte << 23);
#pragma unroll
        for (int q = 0; q < Elem<kType>::kE / 4; ++q) held_values(w.c[q], up, x + 4 * q);
    }
};

// load(places) and then use(i, place, whether it is there) for this block's words,
// kHoldWords a thread at a time.
template <typename Load, typename Use>
__device__ __forceinline__ void each_word(int64_t total, uint32_t words, Load load, Use use) {
    constexpr int64_t kStep = kHoldWords * kBlock;
    for (int64_t first = blockIdx.x * kStep; first < total; first += gridDim.x * kStep) {
        Place at[kHoldWords] = {Place(first, threadIdx.x, words), Place(first, threadIdx.x + kBlock, words),
                                Place(first, threadIdx.x + 2 * kBlock, words),
                                Place(first, threadIdx.x + 3 * kBlock, words)};
        bool in[kHoldWords];
#pragma unroll
        for (int i = 0; i < kHoldWords; ++i) {
            in[i] = first + i * kBlock + threadIdx.x < total;
            if (!in[i]) at[i].row = 0, at[i].word = 0;           // read, not written
        }
        load(at);
#pragma unroll
        for (int i = 0; i < kHoldWords; ++i) use(i, at[i], in[i]);
    }
}
static_assert(kHoldWords == 4, "each_word's places");

// the words at these places of rows x cols values; zeros behind a row's end
template <int kType>
__device__ __forceinline__ void load_places(u32x4 (&v)[kHoldWords], const typename Elem<kType>::T* x,
                                            const Place* p, int64_t cols, int64_t stride, int64_t ld) {
    load_words<kType>(v, cols, cols == ld, [&](int i) { return WordAt<kType>{x + p[i].row * stride, p[i].word}; });
}

template <int kType>
__global__ __launch_bounds__(kBlock) void hold_kernel(const typename Elem<kType>::T* x, int64_t total,
                                                      int64_t cols, int64_t stride, int64_t ld,
                                                      HeldOut<kType> out) {
    u32x4 v[kHoldWords];
    each_word(total, (uint32_t)(ld / Elem<kType>::kE),
              [&](const Place* p) { load_places<kType>(v, x, p, cols, stride, ld); },
              [&](int i, const Place& p, bool in) { out.put(ld, p.row, p.word, v[i], in); });
}

template <int kOut>
__global__ __launch_bounds__(kBlock) void held_values_kernel(HeldIn<kOut> in, int64_t total,
                                                             int64_t cols, int64_t ld,
                                                             typename Elem<kOut>::T* out,
                                                             int64_t stride) {
    typename HeldIn<kOut>::Word w[kHoldWords];
    each_word(total, (uint32_t)(ld / Elem<kOut>::kE),
              [&](const Place* p) {
#pragma unroll
                  for (int i = 0; i < kHoldWords; ++i) w[i] = in.get(ld, p[i].row, p[i].word);
              },
              [&](int i, const Place& p, bool there) {
                  float x[Elem<kOut>::kE];
                  HeldIn<kOut>::values(w[i], x);
                  if (there) store_vec<kOut>(out + p.row * stride, p.word, cols, pack<kOut>(x));
              });
}

// ---- activation functions ------------------------------------------------------------

// f = g s and its slope, s = 1 / (1 + 2^(-z)): z = g log2 e, or 2 u log2 e with
// u = sqrt(2/pi) (g + 0.044715 g^3).  f' = s + g s (1 - s) dz/dg ln 2.
template <int kKind>
__device__ __forceinline__ float share_of(float g) {
    constexpr float kTwoRoot = 1.5957691216057308f;              // 2 sqrt(2/pi)
    const float z = kKind == FLASHOPT_SILU
                        ? g * kLog2e
                        : g * __builtin_fmaf(g * g, kTwoRoot * 0.044715f * kLog2e, kTwoRoot * kLog2e);
    return __builtin_amdgcn_rcpf(1.0f + exp2_hw(-z));
}
template <int kKind>
__device__ __forceinline__ float slope_of(float g, float s) {
    if (kKind == FLASHOPT_SILU) return s * __builtin_fmaf(g, 1.0f - s, 1.0f);
    constexpr float kTwoRoot = 1.5957691216057308f;
    // beyond |g| = 1000 s (1 - s) is 0: the bound keeps 0 * inf out
    const float d = __builtin_fmaf(fminf(g * g, 1e6f), kTwoRoot * 3.0f * 0.044715f, kTwoRoot);
    return __builtin_fmaf(g * s * (1.0f - s), d, s);
}

template <int kType, int kKind, bool kUp>
__global__ __launch_bounds__(kBlock) void gated_kernel(
    const typename Elem<kType>::T* gate, const typename Elem<kType>::T* up, int64_t total,
    int64_t cols, int64_t gate_stride, int64_t up_stride, int64_t ld, typename Elem<kType>::T* y,
    int64_t y_stride, HeldOut<kType> held_gate, HeldOut<kType> held_up) {
    constexpr int E = Elem<kType>::kE;
    u32x4 g[kHoldWords], u[kHoldWords];
    each_word(total, (uint32_t)(ld / E),
              [&](const Place* p) {
                  load_places<kType>(g, gate, p, cols, gate_stride, ld);
                  if (kUp) load_places<kType>(u, up, p, cols, up_stride, ld);
              },
              [&](int i, const Place& p, bool in) {
                  if (held_gate.codes) {
                      held_gate.put(ld, p.row, p.word, g[i], in);
                      if (kUp) held_up.put(ld, p.row, p.word, u[i], in);
                  }
                  if (y && in) {
                      float o[E];
#pragma unroll
                      for (int e = 0; e < E; ++e) {
                          const float x = Elem<kType>::get(g[i], e);
                          o[e] = x * share_of<kKind>(x);
                          if (kUp) o[e] *= Elem<kType>::get(u[i], e);
                      }
                      store_vec<kType>(y + p.row * y_stride, p.word, cols, pack<kType>(o));
                  }
              });
}

template <int kType, int kKind, bool kUp>
__global__ __launch_bounds__(kBlock) void gated_backward_kernel(
    const typename Elem<kType>::T* dy, int64_t total, int64_t cols, int64_t dy_stride, int64_t ld,
    HeldIn<kType> held_gate, HeldIn<kType> held_up, typename Elem<kType>::T* dgate,
    int64_t dgate_stride, typename Elem<kType>::T* dup, int64_t dup_stride) {
    constexpr int E = Elem<kType>::kE;
    u32x4 d[kHoldWords];
    typename HeldIn<kType>::Word wg[kHoldWords], wu[kHoldWords];
    each_word(total, (uint32_t)(ld / E),
              [&](const Place* p) {
#pragma unroll
                  for (int i = 0; i < kHoldWords; ++i) {
                      wg[i] = held_gate.get(ld, p[i].row, p[i].word);
                      if (kUp) wu[i] = held_up.get(ld, p[i].row, p[i].word);
                  }
                  load_places<kType>(d, dy, p, cols, dy_stride, ld);
              },
              [&](int i, const Place& p, bool in) {
                  if (!in) return;
                  float g[E], u[E], a[E], b[E];
                  HeldIn<kType>::values(wg[i], g);
                  if (kUp) HeldIn<kType>::values(wu[i], u);
#pragma unroll
                  for (int e = 0; e < E; ++e) {
                      const float s = share_of<kKind>(g[e]), x = Elem<kType>::get(d[i], e);
                      a[e] = (kUp ? x * u[e] : x) * slope_of<kKind>(g[e], s);
                      if (kUp) b[e] = x * (g[e] * s);
                  }
                  store_vec<kType>(dgate + p.row * dgate_stride, p.word, cols, pack<kType>(a));
                  if (kUp) store_vec<kType>(dup + p.row * dup_stride, p.word, cols, pack<kType>(b));
              });
}

// ---- host ---------------------------------------------------------------------

template <typename F>
static int by_type(int32_t type, F f) {
    if (type == FLASHOPT_BF16) f(std::integral_constant<int, FLASHOPT_BF16>());
    else if (type == FLASHOPT_FP16) f(std::integral_constant<int, FLASHOPT_FP16>());
    else f(std::integral_constant<int, FLASHOPT_FP32>());
    return launch_status();
}

static dim3 word_grid(int64_t total) {
    const int64_t blocks = (total + kHoldWords * kBlock - 1) / (kHoldWords * kBlock);
    return dim3((unsigned)(blocks < kHoldBlocks ? blocks : kHoldBlocks));
}

// a matrix of rows x cols values at p, row stride `stride`
static int check_values(const void* p, int32_t type, int64_t cols, int64_t stride) {
    if (stride < cols || stride > kMaxNumel) return FLASHOPT_ERR_SIZE;
    if (!p) return FLASHOPT_ERR_NULL;
    return aligned(p, type_size(type)) ? FLASHOPT_OK : FLASHOPT_ERR_ALIGN;
}

static int check_shape(int32_t type, int64_t rows, int64_t cols) {
    if (!valid_type(type)) return FLASHOPT_ERR_ARG;
    return rows < 0 || rows > int64_t(1) << 24 || cols < 1 || cols > FLASHOPT_INT8_COLS_MAX
               ? FLASHOPT_ERR_SIZE : FLASHOPT_OK;
}

static int check_held(const void* codes, const void* powers) {
    if (!codes || !powers) return FLASHOPT_ERR_NULL;
    return aligned(codes, 16) ? FLASHOPT_OK : FLASHOPT_ERR_ALIGN;
}

static bool meet(int32_t type, int64_t rows, int64_t cols, const void* a, int64_t a_stride,
                 const void* b, int64_t b_stride) {
    const int64_t size = (int64_t)type_size(type);
    return overlap(rows, a, a_stride * size, cols * size, b, b_stride * size, cols * size);
}

// a matrix and the held arrays of one as large (null: none)
static bool meet_held(int32_t type, int64_t rows, int64_t cols, const void* a, int64_t stride,
                      const void* codes, const void* powers) {
    const int64_t size = (int64_t)type_size(type), held = rows * held_ld(cols);
    return rows_meet(rows, a, (__int128)stride * size, cols * size, codes, held) ||
           rows_meet(rows, a, (__int128)stride * size, cols * size, powers, held / kGroup8);
}

}  // namespace flashopt

using namespace flashopt;

extern "C" {

int64_t flashopt_held_ld(int64_t cols) {
    return cols < 1 || cols > FLASHOPT_INT8_COLS_MAX ? 0 : held_ld(cols);
}

int flashopt_hold(const void* x, int32_t type, int64_t rows, int64_t cols, int64_t stride,
                  int8_t* codes, uint8_t* powers, void* stream) {
    int e = check_shape(type, rows, cols);
    if (e) return e;
    if (stride < cols || stride > kMaxNumel) return FLASHOPT_ERR_SIZE;
    if (rows == 0) return FLASHOPT_OK;
    if ((e = check_values(x, type, cols, stride)) || (e = check_held(codes, powers))) return e;
    if (meet_held(type, rows, cols, x, stride, codes, powers)) return FLASHOPT_ERR_ARG;
    const int64_t ld = held_ld(cols);
    return by_type(type, [&](auto t) {
        constexpr int kType = decltype(t)::value;
        const int64_t total = rows * (ld / Elem<kType>::kE);
        hipLaunchKernelGGL((hold_kernel<kType>), word_grid(total), dim3(kBlock), 0, (hipStream_t)stream,
                           (const typename Elem<kType>::T*)x, total, cols, stride, ld,
                           HeldOut<kType>{codes, powers});
    });
}

int flashopt_held_values(const int8_t* codes, const uint8_t* powers, int64_t rows, int64_t cols,
                         void* out, int32_t type, int64_t out_stride, void* stream) {
    int e = check_shape(type, rows, cols);
    if (e) return e;
    if (out_stride < cols || out_stride > kMaxNumel) return FLASHOPT_ERR_SIZE;
    if (rows == 0) return FLASHOPT_OK;
    if ((e = check_held(codes, powers)) || (e = check_values(out, type, cols, out_stride))) return e;
    if (meet_held(type, rows, cols, out, out_stride, codes, powers)) return FLASHOPT_ERR_ARG;
    const int64_t ld = held_ld(cols);
    return by_type(type, [&](auto t) {
        constexpr int kType = decltype(t)::value;
        const int64_t total = rows * (ld / Elem<kType>::kE);
        hipLaunchKernelGGL((held_values_kernel<kType>), word_grid(total), dim3(kBlock), 0,
                           (hipStream_t)stream, HeldIn<kType>{codes, powers}, total, cols, ld,
                           (typename Elem<kType>::T*)out, out_stride);
    });
}

int flashopt_gated(const void* gate, const void* up, int32_t type, int32_t kind, int64_t rows,
                   int64_t cols, int64_t gate_stride, int64_t up_stride, void* y,
                   int64_t y_stride, int8_t* gate_codes, uint8_t* gate_powers, int8_t* up_codes,
                   uint8_t* up_powers, void* stream) {
    int e = check_shape(type, rows, cols);
    if (e) return e;
    if (kind != FLASHOPT_SILU && kind != FLASHOPT_GELU) return FLASHOPT_ERR_ARG;
    if (rows == 0) return FLASHOPT_OK;
    const bool hold = gate_codes || gate_powers || up_codes || up_powers;
    if (!hold && !y) return FLASHOPT_ERR_NULL;
    if ((e = check_values(gate, type, cols, gate_stride))) return e;
    if (up && (e = check_values(up, type, cols, up_stride))) return e;
    if (hold && (e = check_held(gate_codes, gate_powers))) return e;
    if (hold && up && (e = check_held(up_codes, up_powers))) return e;
    if (!up && (up_codes || up_powers)) return FLASHOPT_ERR_NULL;
    if (y && (e = check_values(y, type, cols, y_stride))) return e;
    if (y && (meet(type, rows, cols, gate, gate_stride, y, y_stride) ||
              (up && meet(type, rows, cols, up, up_stride, y, y_stride))))
        return FLASHOPT_ERR_ARG;
    for (const auto& h : {std::pair<void*, void*>(gate_codes, gate_powers), {up_codes, up_powers}})
        if (meet_held(type, rows, cols, gate, gate_stride, h.first, h.second) ||
            meet_held(type, rows, cols, up, up_stride, h.first, h.second) ||
            meet_held(type, rows, cols, y, y_stride, h.first, h.second))
            return FLASHOPT_ERR_ARG;
    const int64_t ld = held_ld(cols);
    return by_type(type, [&](auto t) {
        constexpr int kType = decltype(t)::value;
        typedef typename Elem<kType>::T T;
        const int64_t total = rows * (ld / Elem<kType>::kE);
        auto with = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, word_grid(total), dim3(kBlock), 0, (hipStream_t)stream,
                               (const T*)gate, (const T*)up, total, cols, gate_stride, up_stride, ld,
                               (T*)y, y_stride, HeldOut<kType>{gate_codes, gate_powers},
                               HeldOut<kType>{up_codes, up_powers});
        };
        if (kind == FLASHOPT_SILU) {
            if (up) with(gated_kernel<kType, FLASHOPT_SILU, true>);
            else with(gated_kernel<kType, FLASHOPT_SILU, false>);
        } else {
            if (up) with(gated_kernel<kType, FLASHOPT_GELU, true>);
            else with(gated_kernel<kType, FLASHOPT_GELU, false>);
        }
    });
}

int flashopt_gated_backward(const void* dy, int32_t type, int32_t kind, int64_t rows, int64_t cols,
                            int64_t dy_stride, const int8_t* gate_codes,
                            const uint8_t* gate_powers, const int8_t* up_codes,
                            const uint8_t* up_powers, void* dgate, int64_t dgate_stride,
                            void* dup, int64_t dup_stride, void* stream) {
    int e = check_shape(type, rows, cols);
    if (e) return e;
    if (kind != FLASHOPT_SILU && kind != FLASHOPT_GELU) return FLASHOPT_ERR_ARG;
    if (rows == 0) return FLASHOPT_OK;
    const bool up = up_codes || up_powers || dup;
    if ((e = check_values(dy, type, cols, dy_stride)) || (e = check_held(gate_codes, gate_powers)) ||
        (e = check_values(dgate, type, cols, dgate_stride)))
        return e;
    if (up && ((e = check_held(up_codes, up_powers)) || (e = check_values(dup, type, cols, dup_stride))))
        return e;
    if (meet(type, rows, cols, dy, dy_stride, dgate, dgate_stride) ||
        (up && (meet(type, rows, cols, dy, dy_stride, dup, dup_stride) ||
                meet(type, rows, cols, dgate, dgate_stride, dup, dup_stride))))
        return FLASHOPT_ERR_ARG;
    if (meet_held(type, rows, cols, dgate, dgate_stride, gate_codes, gate_powers) ||
        meet_held(type, rows, cols, dgate, dgate_stride, up_codes, up_powers) ||
        meet_held(type, rows, cols, dup, dup_stride, gate_codes, gate_powers) ||
        meet_held(type, rows, cols, dup, dup_stride, up_codes, up_powers))
        return FLASHOPT_ERR_ARG;
    const int64_t ld = held_ld(cols);
    return by_type(type, [&](auto t) {
        constexpr int kType = decltype(t)::value;
        typedef typename Elem<kType>::T T;
        const int64_t total = rows * (ld / Elem<kType>::kE);
        auto with = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, word_grid(total), dim3(kBlock), 0, (hipStream_t)stream,
                               (const T*)dy, total, cols, dy_stride, ld,
                               HeldIn<kType>{gate_codes, gate_powers}, HeldIn<kType>{up_codes, up_powers},
                               (T*)dgate, dgate_stride, (T*)dup, dup_stride);
        };
        if (kind == FLASHOPT_SILU) {
            if (up) with(gated_backward_kernel<kType, FLASHOPT_SILU, true>);
            else with(gated_backward_kernel<kType, FLASHOPT_SILU, false>);
        } else {
            if (up) with(gated_backward_kernel<kType, FLASHOPT_GELU, true>);
            else with(gated_backward_kernel<kType, FLASHOPT_GELU, false>);
        }
    });
}

}  // extern "C"
