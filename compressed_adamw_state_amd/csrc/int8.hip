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

constexpr int64_t kLdStep = 128;
static inline int64_t ld_of(int64_t cols) { return (cols + kLdStep - 1) / kLdStep * kLdStep; }

// ---- rounding a row -----------------------------------------------------------

// rne(127 x / a), decided as by exact division.  r = RN(127 / a): x r is within
// 2^-22 of the quotient relative to it, below 2^-15 absolutely, so only a value
// that lies within 2^-12 of a border between two codes needs more: there the
// quotient is formed in binary64, whose rounding error (2^-46 at most here)
// moves it over no border unless an FP32 row holds a value that close to one.
__device__ __forceinline__ int row_code(float x, float a, float r) {
    const float v = x * r;
    float q = __builtin_rintf(v);
    if (__builtin_fabsf(v - q) > 0.5f - 0x1p-12f) q = (float)__builtin_rint((double)x * 127.0 / (double)a);
    return (int)fminf(fmaxf(q, -127.0f), 127.0f);
}

// One block per row; load(j) gives element j as binary32.
template <typename Load>
__device__ __forceinline__ void quantize_row(Load load, int64_t cols, int64_t ld, int8_t* codes,
                                             float* scale) {
    __shared__ float red[kWavesPerBlock];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    // the largest magnitude as an unsigned pattern: infinities and NaN rank above
    uint32_t top = 0;
    for (int64_t j = threadIdx.x; j < cols; j += kBlock)
        top = max(top, as_u32(load(j)) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    if (lane == 0) red[wave] = as_f32(top);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWavesPerBlock; ++w) top = max(top, as_u32(red[w]));
    const bool bad = top >= 0x7F800000u;
    const float a = as_f32(top);
    // a below 2^-100: x r would overflow or be of a subnormal; every code in binary64
    const bool small = a < 0x1p-100f;
    const float r = small || bad ? 0.0f : 127.0f / a;
    for (int64_t j = threadIdx.x; j < ld; j += kBlock) {
        int q = 0;
        if (j < cols && !bad && a > 0.0f) {
            const float x = load(j);
            q = small ? (int)__builtin_rint((double)x * 127.0 / (double)a) : row_code(x, a, r);
        }
        codes[j] = (int8_t)q;
    }
    if (threadIdx.x == 0) *scale = bad ? NAN : a / 127.0f;
}

template <int kType>
__global__ __launch_bounds__(kBlock) void quantize_rows_kernel(const typename Elem<kType>::T* x,
                                                               int64_t cols, int64_t stride,
                                                               int64_t ld, int8_t* codes,
                                                               float* scale) {
    const int64_t row = blockIdx.x;
    const typename Elem<kType>::T* p = x + row * stride;
    quantize_row([&](int64_t j) { return Elem<kType>::up(p[j]); }, cols, ld, codes + row * ld,
                 scale + row);
}

// the same from a tensor's state: the rebuilt master weight, element by element
template <int kOpt, bool kFp32>
__global__ __launch_bounds__(kBlock) void quantize_state_kernel(DevTensor d, int64_t cols,
                                                                int64_t ld, int8_t* codes,
                                                                float* scale) {
    const int64_t row = blockIdx.x;
    const GTensor T = view(d);
    auto load = [&](int64_t j) -> float {
        const int64_t e = row * cols + j;
        if (kFp32) {
            constexpr int F = kOpt == kAdamW ? 3 : 2;
            return ((const GLOBAL float*)T.codes)[(e >> 9) * (512 * F) + (e & 511)];
        }
        return unsplit(T.theta[e], (int32_t)(int8_t)*code_at<kOpt>(T, e, kRho));
    };
    quantize_row(load, cols, ld, codes + row * ld, scale + row);
}

// ---- the product ----------------------------------------------------------------

// One wave per 16 x 16 outputs: v_mfma_i32_16x16x64_i8 with the weight rows as
// its A rows and the tokens as its B columns; lane l holds 16 consecutive
// codes of row l % 16, at (l / 16) * 16, and afterwards the four outputs
// 4 (l / 16) .. + 3 of token l % 16.
template <int kType>
__global__ __launch_bounds__(kBlock) void matmul_kernel(const int8_t* a, const float* a_scale,
                                                        const int8_t* b, const float* b_scale,
                                                        const typename Elem<kType>::T* bias,
                                                        int64_t m, int64_t n, int64_t ld,
                                                        typename Elem<kType>::T* out,
                                                        int64_t out_stride) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t n0 = ((int64_t)blockIdx.x * kWavesPerBlock + wave) * 16;
    const int64_t m0 = (int64_t)blockIdx.y * 16;
    if (n0 >= n) return;
    const int64_t wr = min(n0 + (lane & 15), n - 1), xr = min(m0 + (lane & 15), m - 1);
    const int8_t* w = b + wr * ld + (lane >> 4) * 16;
    const int8_t* x = a + xr * ld + (lane >> 4) * 16;
    i32x4 acc = {0, 0, 0, 0};
    for (int64_t k = 0; k < ld; k += 64)
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(*(const i32x4*)(w + k), *(const i32x4*)(x + k),
                                                    acc, 0, 0, 0);
    const int64_t i = m0 + (lane & 15);
    if (i >= m) return;
    const float s = a_scale[i];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t j = n0 + (lane >> 4) * 4 + r;
        if (j >= n) continue;
        float y = (float)acc[r] * (s * b_scale[j]);
        if (bias) y += Elem<kType>::up(bias[j]);
        out[i * out_stride + j] = Elem<kType>::down(y);
    }
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

static int check_codes(const void* codes, const void* scale) {
    if (!codes || !scale) return FLASHOPT_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scale, 4)) return FLASHOPT_ERR_ALIGN;
    return FLASHOPT_OK;
}

static int launch_quantize(const void* x, int32_t type, int64_t rows, int64_t cols, int64_t stride,
                           int8_t* codes, float* scale, hipStream_t st) {
    return by_type(type, [&](auto k) {
        constexpr int kType = decltype(k)::value;
        hipLaunchKernelGGL((quantize_rows_kernel<kType>), dim3((unsigned)rows), dim3(kBlock), 0, st,
                           (const typename Elem<kType>::T*)x, cols, stride, ld_of(cols), codes,
                           scale);
    });
}

static int launch_matmul(const int8_t* a, const float* a_scale, const int8_t* b,
                         const float* b_scale, const void* bias, int64_t m, int64_t n, int64_t k,
                         void* out, int32_t type, int64_t out_stride, hipStream_t st) {
    return by_type(type, [&](auto t) {
        constexpr int kType = decltype(t)::value;
        typedef typename Elem<kType>::T T;
        const dim3 grid((unsigned)((n + 63) / 64), (unsigned)((m + 15) / 16));
        hipLaunchKernelGGL((matmul_kernel<kType>), grid, dim3(kBlock), 0, st, a, a_scale, b,
                           b_scale, (const T*)bias, m, n, ld_of(k), (T*)out, out_stride);
    });
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
    const dim3 grid((unsigned)rows);
    const int64_t ld = ld_of(cols);
    hipStream_t st = (hipStream_t)stream;
    const bool adam = opt_of(kind) == kAdamW;     // SGD and Lion share a layout
    if (is_fp32(kind)) {
        if (adam) hipLaunchKernelGGL((quantize_state_kernel<kAdamW, true>), grid, dim3(kBlock), 0, st, d, cols, ld, codes, scale);
        else hipLaunchKernelGGL((quantize_state_kernel<kSgd, true>), grid, dim3(kBlock), 0, st, d, cols, ld, codes, scale);
    } else {
        if (adam) hipLaunchKernelGGL((quantize_state_kernel<kAdamW, false>), grid, dim3(kBlock), 0, st, d, cols, ld, codes, scale);
        else hipLaunchKernelGGL((quantize_state_kernel<kSgd, false>), grid, dim3(kBlock), 0, st, d, cols, ld, codes, scale);
    }
    return launch_status();
}

size_t flashopt_int8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (check_matrix(m, k) || check_matrix(n, k)) return 0;
    return up256((size_t)(m * ld_of(k))) + up256((size_t)m * sizeof(float));
}

static int check_product(const int8_t* a, const float* a_scale, const int8_t* b,
                         const float* b_scale, const void* bias, int64_t m, int64_t n, int64_t k,
                         const void* out, int32_t type, int64_t out_stride) {
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
    (void)workspace; (void)workspace_bytes;
    if (!valid_type(out_type)) return FLASHOPT_ERR_ARG;
    if (check_matrix(m, k) || check_matrix(n, k) || out_stride < n || out_stride > kMaxNumel)
        return FLASHOPT_ERR_SIZE;
    if (m == 0 || n == 0) return FLASHOPT_OK;
    const int e = check_product(a, a_scale, b, b_scale, bias, m, n, k, out, out_type, out_stride);
    if (e) return e;
    return launch_matmul(a, a_scale, b, b_scale, bias, m, n, k, out, out_type, out_stride,
                         (hipStream_t)stream);
}

int flashopt_int8_linear(const void* x, int32_t type, int64_t m, int64_t k, int64_t x_stride,
                         const int8_t* w, const float* w_scale, const void* bias, int64_t n,
                         void* out, int64_t out_stride, void* workspace, size_t workspace_bytes,
                         void* stream) {
    if (!valid_type(type)) return FLASHOPT_ERR_ARG;
    if (check_matrix(m, k) || check_matrix(n, k) || out_stride < n || out_stride > kMaxNumel ||
        x_stride < k || x_stride > kMaxNumel)
        return FLASHOPT_ERR_SIZE;
    if (m == 0 || n == 0) return FLASHOPT_OK;
    if (!x || !workspace) return FLASHOPT_ERR_NULL;
    if (!aligned(x, type_size(type))) return FLASHOPT_ERR_ALIGN;
    if (workspace_bytes < flashopt_int8_workspace_bytes(m, n, k) || !aligned(workspace, 256))
        return FLASHOPT_ERR_WORKSPACE;
    int8_t* codes = (int8_t*)workspace;
    float* scale = (float*)((char*)workspace + up256((size_t)(m * ld_of(k))));
    const int e = check_product(codes, scale, w, w_scale, bias, m, n, k, out, type, out_stride);
    if (e) return e;
    const int q = launch_quantize(x, type, m, k, x_stride, codes, scale, (hipStream_t)stream);
    if (q) return q;
    return launch_matmul(codes, scale, w, w_scale, bias, m, n, k, out, type, out_stride,
                         (hipStream_t)stream);
}

}  // extern "C"
