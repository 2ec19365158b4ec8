// Log probabilities of whole rows of logits with their gradient
// (logits.hpp has the mathematics).
//
// A block keeps a row in its registers, kCols 16-byte words a thread, so that
// it is read once and its gradient written once; while the gradient of a
// column of words is stored, the same column of the block's next row is
// loaded into its place.  (The last row's loads have no next row: they read that row
// again and are thrown away.)  Against the segments' code, which reads a row a
// second time from the last-level cache: 4096 x 32000 BF16 94 us for 121 over the same
// logits again and again (105 over four by turns), 1024 x 50257 BF16 50 for 60, 1024 x
// 50257 FP32 100 for 100 (HBM at the rate of a copy: 102, 40, 80).  Rows that would
// need a block of 16 waves, alone on its CU, are left to the segments: nothing else
// runs there between a row's loads and its sums.
//
// What keeps the loop free of waits: every load is unconditional (loads and
// stores come back in order, so a load that a branch may skip would be waited
// for at the branch's end), the words past the row's end read its last word
// again, and addresses are a scalar base per column plus one lane offset.
#include <type_traits>

#include "logits.hpp"

namespace flashopt {

// One block's rows in one call.
template <int kType>
struct RowArgs {
    typedef typename Elem<kType>::T T;
    const T* logits;
    T* grad;
    int64_t rows, stride, grad_stride;
    int32_t vocab;
    float c, inv_t;
    ProbOut out;
    const float *up, *up_entropy;
};

// kEntropy: with the entropy's gradient
template <int kType, int kWaves, int kCols, bool kEntropy>
__global__ __launch_bounds__(kWaves * kWave, 4) void row_kernel(RowArgs<kType> a) {
    constexpr int E = Elem<kType>::kE, kThreads = kWaves * kWave, kSure = kCols - 4;
    constexpr uint32_t kInf = Elem<kType>::kMinusInf;
    typedef typename Elem<kType>::T T;
    __shared__ Part red[kWaves];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int32_t words = a.vocab / E, left = a.vocab % E;       // whole words, entries behind them
    const float c = a.c;

    // The first kSure columns are whole; the others' words may lie past the end.
    u32x4 r[kCols];
    float rest;                                  // of threads 0 .. left - 1
    const uint32_t off = tid * 16u;
    auto at = [&](const T* p, int i) -> GLOBAL char* {
        GLOBAL char* b = (GLOBAL char*)(uint64_t)p + (i < kSure ? i * kThreads * 16 : 0);
        asm volatile("" : "+s"(b));              // one scalar base a column
        const int32_t w = i * kThreads + tid;
        return b + (i < kSure ? off : (uint32_t)min(w, words - 1) * 16u);
    };
    auto load = [&](const T* p, int i) { r[i] = *(const GLOBAL u32x4_any*)at(p, i); };
    auto load_rest = [&](const T* p) {
        rest = Elem<kType>::up(p[tid < left ? words * E + tid : 0]);
    };

    int64_t row = blockIdx.x;
    const T* x = a.logits + row * a.stride;
#pragma unroll
    for (int i = 0; i < kCols; ++i) load(x, i);
    load_rest(x);
    for (;;) {
        const Given t = given_token<kType>(x, a.vocab, row, a.out.targets);
        // entries that are not this row's count as -inf
#pragma unroll
        for (int i = kSure; i < kCols; ++i) {
            const bool in = i * kThreads + tid < words;
#pragma unroll
            for (int q = 0; q < 4; ++q) r[i][q] = in ? r[i][q] : kInf;
        }
        const float z = tid < left ? rest : -INFINITY;

        // a thread's sums, relative to its largest entry
        const float m = fmaxf(z, largest<kType, kCols>(r));
        const float most = m == -INFINITY ? 0.0f : m;
        float u = 0.0f;
        PairSum sum;
        auto one = [&](float v) {
            const float d = (v - most) * c, p = exp2_hw(d);
            u = __builtin_fmaf(p, fmaxf(d, -200.0f), u);
            return p;
        };
        const float first = one(z);
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
            PairSum word;
#pragma unroll
            for (int e = 0; e < E; ++e) word.add(e, one(Elem<kType>::get(r[i], e)));
            sum.add(i, word.total(E));
            asm volatile("" : "+v"(r[i]));       // unpacked again for the gradient, not held
            __builtin_amdgcn_sched_barrier(0);
        }
        const float s = sum.total(kCols) + first;
        const Part p = wave_part<true>(m, s, u, c);
        if (lane == 0) red[wave] = p;
        __syncthreads();
        const Part all = join_parts(red, kWaves, c);

        const int64_t next = row + gridDim.x;
        const bool more = next < a.rows;
        const T* nx = more ? a.logits + next * a.stride : x;     // the last row: loaded, not used
        T* g = a.grad + row * a.grad_stride;
        // value(x): the gradient of an entry that is not the given one
        auto dense = [&](auto value) {
            const float o_rest = value(rest);
#pragma unroll
            for (int i = 0; i < kCols; ++i) {
                float o[E];
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = value(Elem<kType>::get(r[i], e));
                const u32x4 v = pack<kType>(o);
                if (i < kSure) __builtin_nontemporal_store(v, (GLOBAL u32x4_any*)at(g, i));
                else if (i * kThreads + tid < words) __builtin_nontemporal_store(v, (GLOBAL u32x4_any*)at(g, i));
                load(nx, i);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (tid < left) g[words * E + tid] = Elem<kType>::down(o_rest);
            load_rest(nx);
            __syncthreads();                     // the given entry's own comes last
        };
        const ProbStats st = prob_stats(all);
        if (tid == 0) write_prob(row, c, st, t, a.out);
        // 1 / T comes last (without the entropy: in A), so that nothing overflows before
        const float last = kEntropy ? a.inv_t : 1.0f, first_t = kEntropy ? 1.0f : a.inv_t;
        const float gl = t.id >= 0 && st.on != 0.0f && a.up ? a.up[row] * first_t : 0.0f;
        const float gh = kEntropy && st.on != 0.0f ? a.up_entropy[row] : 0.0f;
        const float A = -gl - gh * st.entropy, B = -gh * kLn2, base = st.m, l2 = st.l2s;
        auto value = [&](float v) {
            const float d = __builtin_fmaf(v - base, c, -l2), p = exp2_hw(d);
            return kEntropy ? p * __builtin_fmaf(B, fmaxf(d, -200.0f), A) * last : p * A;
        };
        dense(value);
        if (tid == 0 && t.id >= 0)
            g[t.id] = Elem<kType>::down(given_grad<kEntropy>(t.x, st, c, gl, gh) * last);
        if (!more) break;
        row = next;
        x = nx;
    }
}

// ---- host ---------------------------------------------------------------------

// Rows of up to kWordsShort words are taken here however few they are (one row of
// 16000 in BF16: 5.3 us of the GPU's time for 7.4 in segments, 64 of 32000: 8.2 for
// 11.0); longer ones, which the segments' code cuts over more blocks, from
// kRowsWhole rows on (64 rows of 50257 in BF16: 16.4 us for 10.7, 128: 16.8 for 13.9
// in two launches, from the host 17.8 for 20.4; 200: 17.1 for 21.2).  The least
// columns hold kWordsLeast words.
constexpr int64_t kRowsWhole = 128, kWordsShort = 4096, kWordsLeast = 1024;

template <int kType>
static RowArgs<kType> row_args(const Rows& a, const Upstream& g) {
    RowArgs<kType> r = {};
    typedef typename Elem<kType>::T T;
    r.logits = (const T*)a.logits;
    r.grad = (T*)g.grad;
    r.rows = a.rows;
    r.stride = a.stride;
    r.grad_stride = g.stride;
    r.vocab = (int32_t)a.vocab;
    r.c = (float)(1.4426950408889634073599 / a.temperature);
    r.inv_t = (float)(1.0 / a.temperature);
    r.up = g.logprob;
    r.up_entropy = g.entropy;
    return r;
}

// f(type, waves, columns) for the fewest waves that hold a row, as
// compile-time constants
template <typename F>
static bool by_row(const Rows& a, F f) {
    const int64_t words = a.vocab / (a.type == FLASHOPT_FP32 ? 4 : 8);
    if (words <= kWordsLeast || (words > kWordsShort && a.rows < kRowsWhole)) return false;
    int waves = 4;
    if (words > (int64_t)waves * kWave * 16) waves = 8;
    if (words > (int64_t)waves * kWave * 16) return false;
    const int cols = (int)((words + waves * kWave - 1) / (waves * kWave));
    auto with = [&](auto t) {
        const std::integral_constant<int, 4> w4;
        const std::integral_constant<int, 8> w8;
        const std::integral_constant<int, 12> c12;
        const std::integral_constant<int, 16> c16;
        if (waves == 4) {
            if (cols <= 8) f(t, w4, std::integral_constant<int, 8>());
            else if (cols <= 12) f(t, w4, c12);
            else f(t, w4, c16);
        } else {                                 // more than half of 16 columns
            if (cols <= 12) f(t, w8, c12);
            else f(t, w8, c16);
        }
    };
    if (a.type == FLASHOPT_BF16) with(std::integral_constant<int, FLASHOPT_BF16>());
    else if (a.type == FLASHOPT_FP16) with(std::integral_constant<int, FLASHOPT_FP16>());
    else with(std::integral_constant<int, FLASHOPT_FP32>());
    return true;
}

// Blocks of `waves` waves that the GPU holds at once (4 waves a SIMD), each of
// which then takes every such row.
static dim3 row_grid(int64_t rows, int waves) {
    const int64_t blocks = 256 * 16 / waves;
    return dim3((unsigned)(rows < blocks ? rows : blocks));
}

bool launch_rows_prob(const Rows& a, const ProbOut& out, const Upstream& g, hipStream_t st) {
    return by_row(a, [&](auto t, auto w, auto n) {
        constexpr int kType = decltype(t)::value, kWaves = decltype(w)::value, kCols = decltype(n)::value;
        RowArgs<kType> r = row_args<kType>(a, g);
        r.out = out;
        if (g.entropy)
            hipLaunchKernelGGL((row_kernel<kType, kWaves, kCols, true>), row_grid(a.rows, kWaves),
                               dim3(kWaves * kWave), 0, st, r);
        else
            hipLaunchKernelGGL((row_kernel<kType, kWaves, kCols, false>), row_grid(a.rows, kWaves),
                               dim3(kWaves * kWave), 0, st, r);
    });
}

}  // namespace flashopt
