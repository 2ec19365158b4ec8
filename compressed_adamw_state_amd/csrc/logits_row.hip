// Loss and gradient of whole rows of logits (logits.hpp has the mathematics).
//
// A block keeps a row in its registers, kCols 16-byte words a thread, so that
// it is read once and its gradient written once; while the gradient of a
// column of words is stored, the same column of the block's next row is
// loaded into its place.  Read a second time instead, the rows in flight
// (256 KB each at a vocabulary of 128256 in BF16) no longer fit the last-level
// cache together: 4096 such rows took 651 us, 3.2 GB of traffic for 2.1.
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
    float c, c_low, inv_t;
    DistillIn list;                              // kMode 0
    ProbOut out;                                 // kMode 1, 2 (kMode 0: logprob is the loss)
    const float *up, *up_entropy;
};

// kMode 0: distillation, 1: log probability, 2: log probability and entropy
template <int kType, int kWaves, int kCols, int kMode>
__global__ __launch_bounds__(kWaves * kWave, 4) void row_kernel(RowArgs<kType> a) {
    constexpr int E = Elem<kType>::kE, kThreads = kWaves * kWave, kSure = kCols - 4;
    constexpr bool kList = kMode == 0;
    constexpr uint32_t kInf = Elem<kType>::kMinusInf;
    typedef typename Elem<kType>::T T;
    // kList: a byte for each word of a thread, a bit for each listed entry
    __shared__ __attribute__((aligned(16))) uint8_t marks[kList ? kThreads * 16 : 16];
    __shared__ Part red[kWaves];
    __shared__ ListRow lr;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int32_t words = a.vocab / E, left = a.vocab % E;       // whole words, entries behind them
    const float c = a.c;

    // The first kSure columns are whole; the others' words may lie past the end.
    u32x4 r[kCols];
    float rest;                                  // of threads 0 .. left - 1
    const uint32_t off = tid * 16u;
    auto at = [&](const T* p, int i) -> const char* {
        const char* b = (const char*)p + (i < kSure ? i * kThreads * 16 : 0);
        asm volatile("" : "+s"(b));              // one scalar base a column
        const int32_t w = i * kThreads + tid;
        return b + (i < kSure ? off : (uint32_t)min(w, words - 1) * 16u);
    };
    auto load = [&](const T* p, int i) { r[i] = *reinterpret_cast<const u32x4_any*>(at(p, i)); };
    auto load_rest = [&](const T* p) {
        rest = Elem<kType>::up(p[tid < left ? words * E + tid : 0]);
    };

    int64_t row = blockIdx.x;
    const T* x = a.logits + row * a.stride;
#pragma unroll
    for (int i = 0; i < kCols; ++i) load(x, i);
    load_rest(x);
    if (kList) *reinterpret_cast<u32x4*>(marks + tid * 16) = u32x4{0, 0, 0, 0};
    for (;;) {
        Listed l;
        l.id = -1;
        Given t = {-1, 0.0f};
        bool listed_rest = false;
        if constexpr (kList) {
            __syncthreads();                     // the marks are clear
            if (wave == 0) {
                const ListRow own = list_row<kType>(x, a.vocab, row, c, a.list, l);
                const int w = l.id / E;
                if (l.id >= 0 && w < words) {
                    const uint32_t byte = (w % kThreads) * 16 + w / kThreads;
                    atomicOr((uint32_t*)marks + byte / 4, 1u << (byte % 4 * 8 + l.id % E));
                }
                // the entries behind the words are wave 0's own
                for (int k = 0; k < a.list.top; ++k)
                    listed_rest |= __builtin_amdgcn_readlane(l.id, k) == words * E + tid;
                if (lane == 0) lr = own;
            }
            __syncthreads();
        } else {
            t = given_token<kType>(x, a.vocab, row, a.out.targets);
        }
        const bool has_rest = tid < left && !listed_rest;
        // entries that are not this row's, or are listed, count as -inf
#pragma unroll
        for (int i = kSure; i < kCols; ++i) {
            const bool in = i * kThreads + tid < words;
#pragma unroll
            for (int q = 0; q < 4; ++q) r[i][q] = in ? r[i][q] : kInf;
        }
        if constexpr (kList) {
            const u32x4 mine = *reinterpret_cast<const u32x4*>(marks + tid * 16);
            if (mine[0] | mine[1] | mine[2] | mine[3]) {
#pragma unroll
                for (int i = 0; i < kCols; ++i) {
                    const uint32_t bits = mine[i / 4] >> (i % 4 * 8) & 0xFFu;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t mask;
                        if (kType == FLASHOPT_FP32) mask = 0u - (bits >> q & 1u);
                        else mask = ((0u - (bits >> (2 * q) & 1u)) & 0xFFFFu) | ((0u - (bits >> (2 * q + 1) & 1u)) << 16);
                        r[i][q] = (r[i][q] & ~mask) | (kInf & mask);
                    }
                }
            }
        }
        const float z = has_rest ? rest : -INFINITY;

        // A thread's sums, with the maximum of its first words as the shift; if
        // others exceed it by 2^24, once more with the maximum of all.
        float m = z, s, u;
        auto most = [&](int from, int to) {
#pragma unroll
            for (int i = 0; i < kCols; ++i)
                if (i >= from && i < to)
#pragma unroll
                    for (int e = 0; e < E; ++e) m = fmaxf(m, Elem<kType>::get(r[i], e));
        };
        auto sums = [&]() {
            const float base = m == -INFINITY ? 0.0f : m;
            s = u = 0.0f;
            auto one = [&](float v) {
                const float d = (v - base) * c, p = exp2_hw(d);
                s += p;
                if (!kList) u = __builtin_fmaf(p, fmaxf(d, -200.0f), u);
            };
            one(z);
#pragma unroll
            for (int i = 0; i < kCols; ++i) {
#pragma unroll
                for (int e = 0; e < E; ++e) one(Elem<kType>::get(r[i], e));
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        most(0, 2);
        sums();
        if (m == -INFINITY || !(s < 0x1p24f)) {
#pragma unroll
            for (int i = 0; i < kCols; ++i) asm volatile("" : "+v"(r[i]));
            most(0, kCols);
#pragma unroll
            for (int i = 0; i < kCols; ++i) asm volatile("" : "+v"(r[i]));
            sums();
        }
        const Part p = wave_part<!kList>(m, s, u, c);
        if (lane == 0) red[wave] = p;
        __syncthreads();
        const Part all = join_parts(red, kWaves, c);

        const int64_t next = row + gridDim.x;
        const bool more = next < a.rows;
        const T* nx = more ? a.logits + next * a.stride : x;     // the last row: loaded, not used
        T* g = a.grad + row * a.grad_stride;
        // value(x): the gradient of an entry that is not listed or given
        auto dense = [&](auto value) {
            const float o_rest = value(rest);
#pragma unroll
            for (int i = 0; i < kCols; ++i) {
                float o[E];
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = value(Elem<kType>::get(r[i], e));
                const u32x4 v = pack<kType>(o);
                if (i < kSure) *reinterpret_cast<u32x4_any*>(const_cast<char*>(at(g, i))) = v;
                else if (i * kThreads + tid < words) *reinterpret_cast<u32x4_any*>(const_cast<char*>(at(g, i))) = v;
                load(nx, i);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (tid < left) g[words * E + tid] = Elem<kType>::down(o_rest);
            load_rest(nx);
            __syncthreads();                     // the listed or given entries' own come last
        };
        if constexpr (kList) {
            *reinterpret_cast<u32x4*>(marks + tid * 16) = u32x4{0, 0, 0, 0};
            float* loss = a.out.logprob;
            const DistillStats st = finish_row(all, lr, a.list.tail, c, a.c_low, l, row, loss, nullptr, true);
            const float w = st.on != 0.0f ? a.up[row] * a.inv_t : 0.0f;
            const float k = w * st.coef, base = st.rest_m, l2 = st.rest_l2;
            dense([&](float v) { return k * exp2_hw(__builtin_fmaf(v - base, c, -l2)); });
            if (wave == 0) {
                const float v = listed_grad(l, st, a.list.top, c, w);
                if (l.id >= 0) g[l.id] = Elem<kType>::down(v);
            }
        } else {
            const ProbStats st = prob_stats(all);
            if (tid == 0) write_prob(row, c, st, t, a.out);
            const float gl = t.id >= 0 && st.on != 0.0f && a.up ? a.up[row] * a.inv_t : 0.0f;
            const float gh = kMode == 2 ? a.up_entropy[row] * a.inv_t : 0.0f;
            const float A = -gl - gh * st.entropy, B = -gh * kLn2, base = st.m, l2 = st.l2s;
            auto value = [&](float v) {
                const float d = __builtin_fmaf(v - base, c, -l2), p = exp2_hw(d);
                return p * (kMode == 2 ? __builtin_fmaf(B, fmaxf(d, -200.0f), A) : A);
            };
            dense(value);
            if (tid == 0 && t.id >= 0) g[t.id] = Elem<kType>::down(value(t.x) + gl);
        }
        if (!more) break;
        row = next;
        x = nx;
    }
}

// ---- host ---------------------------------------------------------------------

// Rows from which a block a row is worth it, and words of a row.
constexpr int64_t kRowsWhole = 128, kWordsLeast = 1024;

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
    const double c = 1.4426950408889634073599 / a.temperature;
    r.c = (float)c;
    r.c_low = (float)(c - (double)r.c);
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
    if (a.rows < kRowsWhole || words <= kWordsLeast) return false;
    int waves = 4;
    while (waves < 16 && words > (int64_t)waves * kWave * 16) waves *= 2;
    if (words > (int64_t)waves * kWave * 16) return false;
    const int cols = (int)((words + waves * kWave - 1) / (waves * kWave));
    auto with = [&](auto t) {
        auto by_cols = [&](auto w) {
            if (cols <= 8) f(t, w, std::integral_constant<int, 8>());
            else if (cols <= 12) f(t, w, std::integral_constant<int, 12>());
            else f(t, w, std::integral_constant<int, 16>());
        };
        if (waves == 4) by_cols(std::integral_constant<int, 4>());
        else if (waves == 8) by_cols(std::integral_constant<int, 8>());
        else by_cols(std::integral_constant<int, 16>());
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
            hipLaunchKernelGGL((row_kernel<kType, kWaves, kCols, 2>), row_grid(a.rows, kWaves),
                               dim3(kWaves * kWave), 0, st, r);
        else
            hipLaunchKernelGGL((row_kernel<kType, kWaves, kCols, 1>), row_grid(a.rows, kWaves),
                               dim3(kWaves * kWave), 0, st, r);
    });
}

bool launch_rows_distill(const Rows& a, const DistillIn& list, float* loss, const Upstream& g,
                         hipStream_t st) {
    return by_row(a, [&](auto t, auto w, auto n) {
        constexpr int kType = decltype(t)::value, kWaves = decltype(w)::value, kCols = decltype(n)::value;
        RowArgs<kType> r = row_args<kType>(a, g);
        r.list = list;
        r.out.logprob = loss;
        hipLaunchKernelGGL((row_kernel<kType, kWaves, kCols, 0>), row_grid(a.rows, kWaves),
                           dim3(kWaves * kWave), 0, st, r);
    });
}

}  // namespace flashopt
