// Rows of logits (include/flashopt_lm.h): log probabilities of given tokens
// with entropy and top alternatives, distillation from a teacher's top
// logits, and their gradients.
//
// Mathematics.  With c = log2(e) / T and any shift m, a row's distribution is
// p_j = 2^((x_j - m) c) / S, S = sum_j 2^((x_j - m) c).  Each work item (a
// block, over one chunk of one row held in registers) forms the chunk's own
// maximum m and sums
//   S = sum_j e_j,  U = sum_j e_j d_j   (d_j = (x_j - m) c, e_j = 2^d_j);
// a join over the row's chunks rescales them to the row's maximum:
//   S = sum S_c 2^(D_c),  U = sum 2^(D_c) (U_c + D_c S_c),  D_c = (m_c - m) c.
// Then log2 p_j = d_j - log2 S and H = ln2 (log2 S - U / S), both without
// cancellation.  The difference x - m is formed before the scaling, so that
// entries of the type's lowest value stay finite and a row of nothing else is
// uniform.
//
// The gradients are elementwise in the row's numbers: one more pass over the
// chunks, plus a few entries (the given token, the teacher's alternatives)
// that the chunk's block writes again after its dense pass, from logits it
// read before it, so that a gradient may replace its logits.
#include <cmath>

#include "rows.hpp"

namespace flashopt {

// 16-byte words of a chunk per thread: 8 streams best; with few rows 2 give
// more, shorter work items.
constexpr int kLong = 8, kShort = 2;
template <int kType, int kVecs> constexpr int kChunk = kVecs * kBlock * Elem<kType>::kE;

// A part of a row: maximum of x, S, U.
struct Part {
    float m, s, u, pad;
};

// A row's order of entries as unsigned numbers: larger logit first, equal
// ones by lowest id; a NaN ranks above all.
__device__ __forceinline__ uint32_t value_key(float x) {
    uint32_t b = as_u32(x);
    const uint32_t mag = b & 0x7FFFFFFFu;
    if (mag > 0x7F800000u) return 0xFFFFFFFFu;
    if (mag == 0) b = 0;                         // -0 equals +0
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return as_f32((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ uint64_t entry(float x, uint32_t id) {
    return ((uint64_t)value_key(x) << 32) | (0xFFFFFFFFu - id);   // never 0 for an id that exists
}
__device__ __forceinline__ uint32_t entry_id(uint64_t e) { return 0xFFFFFFFFu - (uint32_t)e; }
__device__ __forceinline__ uint32_t entry_key(uint64_t e) { return (uint32_t)(e >> 32); }

// A segment of a row: the words [begin, end) of 16 bytes; the row's last
// word may be partial.
template <int kType>
struct Segment {
    typedef typename Elem<kType>::T T;
    const T* x;
    int64_t vocab, begin, end;                   // words
    int64_t row;

    template <int kVecs>
    __device__ __forceinline__ void load(int64_t chunk, u32x4* r) const {
        const int64_t v0 = begin + chunk * (kVecs * kBlock);
        if (whole<kVecs>(v0)) {                  // all loads in flight at once
            const T* p = x + v0 * Elem<kType>::kE;
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                r[i] = *reinterpret_cast<const u32x4_any*>(p + (threadIdx.x + i * kBlock) * Elem<kType>::kE);
        } else {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int64_t w = v0 + threadIdx.x + i * kBlock;
                // words past the segment belong to another block, or to no row
                r[i] = load_vec<kType>(x, w, w < end ? vocab : 0, Elem<kType>::kMinusInf);
            }
        }
    }
    // a chunk of whole words, all of the segment (equal for the block's threads)
    template <int kVecs>
    __device__ __forceinline__ bool whole(int64_t v0) const {
        const int64_t e = v0 + kVecs * kBlock;
        return e <= end && e * Elem<kType>::kE <= vocab;
    }
    template <int kVecs>
    __device__ __forceinline__ void store(T* g, int64_t chunk, int i, u32x4 o) const {
        const int64_t v0 = begin + chunk * (kVecs * kBlock);
        if (whole<kVecs>(v0)) {
            *reinterpret_cast<u32x4_any*>(g + v0 * Elem<kType>::kE + (threadIdx.x + i * kBlock) * Elem<kType>::kE) = o;
        } else {
            const int64_t w = v0 + threadIdx.x + i * kBlock;
            store_vec<kType>(g, w, w < end ? vocab : 0, o);
        }
    }
    template <int kVecs>
    __device__ __forceinline__ int chunks() const {
        return (int)((end - begin + kVecs * kBlock - 1) / (kVecs * kBlock));
    }
    __device__ __forceinline__ int64_t first_id() const { return begin * Elem<kType>::kE; }
    __device__ __forceinline__ int64_t end_id() const {
        const int64_t e = end * Elem<kType>::kE;
        return e < vocab ? e : vocab;
    }
};

// ---- the best entries of a segment ----------------------------------------------

constexpr int kFound = 512;                      // candidates kept before the exact search is taken

struct TopShared {
    float best[kBlock];                          // each thread's largest entry
    uint64_t found[kFound];
    uint32_t nfound, count[2][kWavesPerBlock];
};

// The `need` best entries into found[0, need), whatever the values: an entry
// is its value and id as one number, so all differ, and the bits of the
// need-th largest are set from the highest down, counting the entries at or
// above each trial.  One pass over the segment a bit: the path of rows with
// hundreds of equal entries at the border or with NaN.
template <int kType, int kVecs>
__device__ __noinline__ void search_top(const Segment<kType>& seg, uint32_t need, TopShared& sh) {
    constexpr int E = Elem<kType>::kE;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int nchunk = seg.template chunks<kVecs>();
    auto each = [&](auto f) {
        for (int ch = 0; ch < nchunk; ++ch) {
            u32x4 r[kVecs];
            seg.template load<kVecs>(ch, r);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int64_t w = seg.begin + ((int64_t)ch * kVecs + i) * kBlock + threadIdx.x;
                if (w < seg.end)
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (w * E + e < seg.vocab)
                            f(entry(Elem<kType>::get(r[i], e), (uint32_t)(w * E + e)));
            }
        }
    };
    uint64_t bound = 0;
    int turn = 0;
    __syncthreads();
    for (int bit = 63; bit >= 0; --bit) {
        if (bit < 32 && bit >= 20) {             // ids are below 2^20: these bits are set
            bound |= uint64_t(1) << bit;
            continue;
        }
        const uint64_t trial = bound | (uint64_t(1) << bit);
        uint32_t n = 0;
        each([&](uint64_t x) { n += x >= trial ? 1u : 0u; });
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) n += __shfl_xor((int)n, o);
        if (lane == 0) sh.count[turn][wave] = n;
        __syncthreads();
        uint32_t all = 0;
#pragma unroll
        for (int w = 0; w < kWavesPerBlock; ++w) all += sh.count[turn][w];
        turn ^= 1;
        if (all >= need) bound = trial;
    }
    if (threadIdx.x == 0) sh.nfound = 0;
    __syncthreads();
    each([&](uint64_t x) {
        if (x >= bound) {
            const uint32_t at = atomicAdd(&sh.nfound, 1u);
            if (at < (uint32_t)kFound) sh.found[at] = x;
        }
    });
    __syncthreads();
}

// The `top` best entries of a segment, best first, through out(rank, entry);
// ranks past the segment's entries get 0.  chunk_best[ch * kBlock + t] holds
// thread t's largest entry of chunk ch, `mine` its largest of all.
//
// The top-th largest of the threads' own maxima is a lower bound of the
// top-th largest entry (that many threads hold an entry at or above it), and
// close to it: the entries lie over the threads by turns, so about
// -256 ln(1 - top/256) of them, 74 for 64, are at or above it.  Only the
// chunks whose maximum is at or above it are read again, by their thread.
template <int kType, int kVecs, typename Out>
__device__ __forceinline__ void segment_top(const Segment<kType>& seg, const float* chunk_best,
                                            float mine, int top, TopShared& sh, Out out) {
    constexpr int E = Elem<kType>::kE;
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t entries = seg.end_id() - seg.first_id();
    const uint32_t need = entries < top ? (uint32_t)entries : (uint32_t)top;
    sh.best[threadIdx.x] = mine;
    if (threadIdx.x == 0) sh.nfound = 0;
    __syncthreads();
    // the bound's upper 16 bits, from the highest down (every wave for itself)
    uint32_t k[kWavesPerBlock], bound = 0;
#pragma unroll
    for (int j = 0; j < kWavesPerBlock; ++j) k[j] = value_key(sh.best[lane + j * kWave]) >> 16;
#pragma unroll
    for (int bit = 15; bit >= 0; --bit) {
        const uint32_t trial = bound | (1u << bit);
        int n = 0;
#pragma unroll
        for (int j = 0; j < kWavesPerBlock; ++j) n += __popcll(__ballot(k[j] >= trial));
        if (n >= top) bound = trial;
    }
    // 0x007F: -inf.  Fewer than `top` threads hold a finite entry: take those,
    // and fill up with entries of -inf
    const bool few = bound <= 0x007Fu;
    const float low = few ? -INFINITY : key_value(bound << 16);
    const int nchunk = seg.template chunks<kVecs>();
    for (int ch = 0; ch < nchunk; ++ch) {
        const float b = chunk_best[ch * kBlock + threadIdx.x];
        if (few ? b > low : b >= low) {
            u32x4 r[kVecs];
            seg.template load<kVecs>(ch, r);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int64_t w = seg.begin + ((int64_t)ch * kVecs + i) * kBlock + threadIdx.x;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float x = Elem<kType>::get(r[i], e);
                    if (few ? x > low : x >= low) {      // padding is -inf, never taken
                        const uint32_t at = atomicAdd(&sh.nfound, 1u);
                        if (at < (uint32_t)kFound) sh.found[at] = entry(x, (uint32_t)(w * E + e));
                    }
                }
            }
        }
    }
    __syncthreads();
    uint32_t n = sh.nfound;
    if (few && n < need) {
        // the lowest ids that hold -inf are among the first n + need
        __syncthreads();
        if (threadIdx.x < kWave) {
            uint32_t have = n;
            for (uint32_t j = 0; j < n + need && have < need; j += kWave) {
                const int64_t id = seg.first_id() + j + lane;
                const bool is = j + lane < n + need && id < seg.end_id() &&
                                Elem<kType>::up(seg.x[id]) == -INFINITY;
                const uint64_t who = __ballot(is);
                const uint32_t at = have + __popcll(who & ((uint64_t(1) << lane) - 1));
                if (is && at < need) sh.found[at] = entry(-INFINITY, (uint32_t)id);
                have += __popcll(who);
            }
            if (lane == 0) sh.nfound = have < need ? have : need;
        }
        __syncthreads();
        n = sh.nfound;
    }
    if (n < need || n > (uint32_t)kFound) {      // equal for all threads
        search_top<kType, kVecs>(seg, need, sh);
        n = need;
    }
    for (uint32_t t = threadIdx.x; t < n; t += kBlock) {
        const uint64_t x = sh.found[t];
        uint32_t rank = 0;
        for (uint32_t j = 0; j < n; ++j) rank += sh.found[j] > x ? 1u : 0u;
        if (rank < need) out(rank, x);
    }
    if (threadIdx.x >= need && threadIdx.x < (uint32_t)top) out(threadIdx.x, uint64_t(0));
}

// ---- a row's numbers --------------------------------------------------------------

// The row's part from its segments' (one wave; every lane gets it).
__device__ __forceinline__ Part join_parts(const Part* part, int n, float c) {
    const int lane = threadIdx.x & (kWave - 1);
    float m = -INFINITY;
    for (int k = lane; k < n; k += kWave) m = fmaxf(m, part[k].m);
    m = wave_max(m);
    float s = 0.0f, u = 0.0f;
    for (int k = lane; k < n; k += kWave) {
        const Part p = part[k];
        if (p.m == -INFINITY && p.s == 0.0f) continue;           // an empty part
        const float D = fmaxf((p.m - m) * c, -200.0f), f = exp2_hw(D);
        s += p.s * f;
        u += f * (p.u + D * p.s);
    }
    return Part{m, wave_sum(s), wave_sum(u), 0.0f};
}

// stats of a row for the gradient: shift m, log2 S, H, and whether the row has
// a distribution (1 or 0).  One without keeps shift 0, so that its entries
// give 2^(-inf) = 0.
struct ProbStats {
    float m, l2s, entropy, on;
};

__device__ __forceinline__ ProbStats prob_stats(const Part& p) {
    const bool empty = p.m == -INFINITY && p.s == 0.0f;
    ProbStats st;
    st.m = empty ? 0.0f : p.m;
    st.l2s = empty ? 0.0f : log2_hw(p.s);
    st.entropy = empty ? 0.0f : (st.l2s - p.u / p.s) * kLn2;
    st.on = empty ? 0.0f : 1.0f;
    return st;
}

struct ProbOut {                                 // each may be null
    const int64_t* targets;
    float *logprob, *entropy;
    ProbStats* stats;
    float* top_logprob;
    int64_t* top_id;
};

// one lane
template <int kType>
__device__ __forceinline__ void write_prob(const typename Elem<kType>::T* x, int64_t vocab,
                                           int64_t row, float c, const ProbStats& st,
                                           const ProbOut& o) {
    if (o.entropy) o.entropy[row] = st.entropy;
    if (o.stats) o.stats[row] = st;
    if (o.logprob) {
        const int64_t t = o.targets[row];
        float lp = 0.0f;
        if (t >= 0 && t < vocab) lp = ((Elem<kType>::up(x[t]) - st.m) * c - st.l2s) * kLn2;
        o.logprob[row] = lp;
    }
}
__device__ __forceinline__ void write_top(const ProbOut& o, int64_t row, int top, int k,
                                          uint64_t e, float c, const ProbStats& st) {
    o.top_id[row * top + k] = entry_id(e);
    o.top_logprob[row * top + k] = ((key_value(entry_key(e)) - st.m) * c - st.l2s) * kLn2;
}

// stats of a row of distillation.  The gradient is
//   outside the list: e_j coef, e_j = 2^((x_j - rest_m) c - rest_l2) the
//                     entry's share of the rest, coef = (Q + r) P - r;
//   in the list:      (Q + r) p_j - sum of its q, p_j from m and l2s;
// q_k = 2^(t_k log2e - norm), all times g / T.  A row without a gradient has
// on = 0.
struct DistillStats {
    float rest_m, rest_l2, coef, qr, m, l2s, norm, on;
};

struct DistillIn {
    const int64_t* ids;
    const float* tlp;
    int top, tail;
};

// log2 of s as a whole number and the rest, which is then off by 2^-24 or so
// whatever the size of s
__device__ __forceinline__ void log2_parts(float s, float& whole, float& frac) {
    const int e = __builtin_amdgcn_frexp_expf(s);
    whole = (float)e;
    frac = log2_hw(__builtin_amdgcn_ldexpf(s, -e));
}
// a * b as a rounded product and its rounding error, plus a * b_low
__device__ __forceinline__ void product_parts(float a, float b, float b_low, float& hi, float& lo) {
    hi = a * b;
    lo = __builtin_fmaf(a, b, -hi) + a * b_low;
}
constexpr float kLog2eLow = 0x1.4ae0cp-26f;      // 1 / log 2 - kLog2e

// q = 2^(t log2e - norm) with norm = whole + frac: the whole part goes into
// the exponent, so that q is good to its last bits for small q too
__device__ __forceinline__ float teacher_q(float t, float nwhole, float nfrac, float& hi, float& lo) {
    product_parts(t, kLog2e, kLog2eLow, hi, lo);
    if (!(hi > -300.0f)) { lo = 0.0f; return t != t ? t : 0.0f; }
    const float n = __builtin_rintf(hi);
    return __builtin_amdgcn_ldexpf(exp2_hw((hi - n) + (lo - nfrac)), (int)(n - nwhole));
}

// The row's loss and stats from the part of its unlisted entries (one wave).
// The divergence is a difference of logarithms near 10 that may itself be
// near 0: their whole parts are subtracted exactly.
template <int kType>
__device__ __forceinline__ DistillStats distill_stats(const typename Elem<kType>::T* x,
                                                      int64_t vocab, int64_t row, float c,
                                                      float c_low, const DistillIn& in,
                                                      const Part& rest, float& loss) {
    const int lane = threadIdx.x & (kWave - 1);
    // lane k holds alternative k; a repeated id is summed into S once
    const int64_t id = lane < in.top ? in.ids[row * in.top + lane] : -1;
    const bool ok = id >= 0 && id < vocab;
    const int own = ok ? (int)id : -1;
    const float xk = ok ? Elem<kType>::up(x[id]) : -INFINITY;
    const float t = ok ? in.tlp[row * in.top + lane] : -INFINITY;
    bool first = ok;
    for (int k = 0; k < in.top - 1; ++k) {
        const int other = __builtin_amdgcn_readlane(own, k);
        if (k < lane && other == own) first = false;
    }
    const float m0 = fmaxf(rest.m, wave_max(xk));
    const bool no_rest = rest.m == -INFINITY && rest.s == 0.0f;
    // the student's row has no distribution
    const bool empty = m0 == -INFINITY && no_rest && __ballot(ok && xk != xk) == 0;
    const float m = empty ? 0.0f : m0;
    const float rest_f = no_rest ? 0.0f : exp2_hw(fmaxf((rest.m - m) * c, -200.0f));
    const float s = wave_sum(first ? exp2_hw((xk - m) * c) : 0.0f) + (no_rest ? 0.0f : rest.s * rest_f);
    float sw = 0.0f, sf = 0.0f, rw = 0.0f, rf = 0.0f;
    if (!empty) log2_parts(s, sw, sf);
    if (!no_rest) log2_parts(rest.s, rw, rf);
    // the teacher's side
    float nw = 0.0f, nf = 0.0f;
    if (!in.tail) {
        const float tm = wave_max(t);
        const float ts = wave_sum(ok ? exp2_hw((t - tm) * kLog2e) : 0.0f);
        float hi, lo, w, f;
        product_parts(tm, kLog2e, kLog2eLow, hi, lo);
        log2_parts(ts, w, f);
        const float n = __builtin_rintf(hi);
        nw = n + w;
        nf = (hi - n) + (lo + f);
    }
    float hi, lo;
    const float q = ok ? teacher_q(t, nw, nf, hi, lo) : 0.0f;
    const float Q = wave_sum(q);
    float r = in.tail ? fmaxf(0.0f, 1.0f - Q) : 0.0f;
    if (no_rest) r = 0.0f;
    // log2 q - log2 p
    float term = 0.0f;
    if (q > 0.0f) {
        float ph, pl;
        product_parts(xk - m, c, c_low, ph, pl);
        if (!(ph > -3e38f)) pl = 0.0f;
        term = q * (((hi - ph) + (sw - nw)) + ((lo - pl) + (sf - nf)));
    } else if (q != 0.0f) {
        term = q;                                // NaN
    }
    float sum = wave_sum(term);
    const float rest_m = no_rest ? 0.0f : rest.m;
    float dh, dl;
    product_parts(rest_m - m, c, c_low, dh, dl);
    if (!(dh > -3e38f)) dl = 0.0f;
    if (r > 0.0f) {
        float w, f;
        log2_parts(r, w, f);
        sum += r * (((w - rw) + sw - dh) + ((f - rf) + (sf - dl)));
    }
    const float P = no_rest ? 0.0f : exp2_hw((dh + (rw - sw)) + (dl + (rf - sf)));
    const bool on = __ballot(ok) != 0 && !empty;
    loss = on ? sum * kLn2 : 0.0f;
    return DistillStats{rest_m, rw + rf, on ? (Q + r) * P - r : 0.0f, Q + r, m, sw + sf, nw + nf,
                        on ? 1.0f : 0.0f};
}

// ---- gradients --------------------------------------------------------------------

// grad_j = p_j (A + B d_j) with d_j = log2 p_j, plus gl at the given token.
template <int kType>
struct ProbGrad {
    const float *grad_logprob, *grad_entropy;    // either may be null
    typename Elem<kType>::T* grad;
    int64_t stride;
    float inv_t;
};

// One chunk of the gradient; target < 0: none.
template <int kType, int kVecs, bool kEntropy>
__device__ __forceinline__ void prob_grad_chunk(const Segment<kType>& seg, int ch, float c, float A,
                                                float B, const ProbStats& st,
                                                typename Elem<kType>::T* g) {
    constexpr int E = Elem<kType>::kE;
    u32x4 r[kVecs];
    seg.template load<kVecs>(ch, r);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float d = (Elem<kType>::get(r[i], e) - st.m) * c - st.l2s;
            const float p = exp2_hw(d);
            o[e] = p * (kEntropy ? __builtin_fmaf(B, fmaxf(d, -200.0f), A) : A);
        }
        seg.template store<kVecs>(g, ch, i, pack<kType>(o));
    }
}

template <int kType, int kVecs, bool kEntropy>
__device__ __forceinline__ void prob_grad_segment(const Segment<kType>& seg, float c,
                                                  const ProbStats& st, const int64_t* targets,
                                                  const ProbGrad<kType>& G) {
    typename Elem<kType>::T* g = G.grad + seg.row * G.stride;
    const int64_t t = targets ? targets[seg.row] : -1;
    const bool given = t >= seg.first_id() && t < seg.end_id();
    const bool in_row = t >= 0 && t < seg.vocab && st.on != 0.0f;
    const float gl = in_row && G.grad_logprob ? G.grad_logprob[seg.row] * G.inv_t : 0.0f;
    const float gh = kEntropy ? G.grad_entropy[seg.row] * G.inv_t : 0.0f;
    const float A = -gl - gh * st.entropy, B = -gh * kLn2;
    float at_t = 0.0f;
    if (given && threadIdx.x == 0) {
        const float d = (Elem<kType>::up(seg.x[t]) - st.m) * c - st.l2s;
        at_t = exp2_hw(d) * (kEntropy ? __builtin_fmaf(B, fmaxf(d, -200.0f), A) : A) + gl;
    }
    __syncthreads();                             // read before a gradient that replaces it is written
    const int n = seg.template chunks<kVecs>();
    for (int ch = 0; ch < n; ++ch) prob_grad_chunk<kType, kVecs, kEntropy>(seg, ch, c, A, B, st, g);
    __syncthreads();                             // after the dense pass's write of the same entry
    if (given && threadIdx.x == 0) g[t] = Elem<kType>::down(at_t);
}

template <int kType>
struct DistillGrad {
    const float* grad_loss;
    typename Elem<kType>::T* grad;
    int64_t stride;
    float inv_t;
};

template <int kType, int kVecs>
__device__ __forceinline__ void distill_grad_segment(const Segment<kType>& seg, float c,
                                                     const DistillStats& st, const DistillIn& in,
                                                     const DistillGrad<kType>& G) {
    constexpr int E = Elem<kType>::kE;
    typename Elem<kType>::T* g = G.grad + seg.row * G.stride;
    const float w = st.on != 0.0f ? G.grad_loss[seg.row] * G.inv_t : 0.0f;
    // wave 0 forms the listed entries' gradients before any gradient is written
    int64_t id = -1;
    float listed = 0.0f;
    if (threadIdx.x < kWave) {
        const int lane = threadIdx.x;
        id = lane < in.top ? in.ids[seg.row * in.top + lane] : -1;
        const bool ok = id >= 0 && id < seg.vocab;
        const float nw = __builtin_rintf(st.norm);
        float hi, lo;
        const float q = ok ? teacher_q(in.tlp[seg.row * in.top + lane], nw, st.norm - nw, hi, lo) : 0.0f;
        if (!ok) id = -1;
        float sum = 0.0f;
        for (int k = 0; k < in.top; ++k) {
            const int other = __builtin_amdgcn_readlane((int)id, k);
            const float oq = as_f32((uint32_t)__builtin_amdgcn_readlane((int)as_u32(q), k));
            if (other == (int)id) sum += oq;
        }
        if (id < seg.first_id() || id >= seg.end_id()) id = -1;
        if (id >= 0) {
            const float p = exp2_hw((Elem<kType>::up(seg.x[id]) - st.m) * c - st.l2s);
            listed = st.on != 0.0f ? w * (st.qr * p - sum) : 0.0f;
        }
    }
    __syncthreads();
    const float a = w * st.coef;
    const int n = seg.template chunks<kVecs>();
    for (int ch = 0; ch < n; ++ch) {
        u32x4 r[kVecs];
        seg.template load<kVecs>(ch, r);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            float o[E];
#pragma unroll
            for (int e = 0; e < E; ++e)
                o[e] = a * exp2_hw((Elem<kType>::get(r[i], e) - st.rest_m) * c - st.rest_l2);
            seg.template store<kVecs>(g, ch, i, pack<kType>(o));
        }
    }
    __syncthreads();
    if (id >= 0) g[id] = Elem<kType>::down(listed);
}

// ---- kernels ------------------------------------------------------------------------

// Rows cut into nseg segments of `span` words each; one block per segment.
template <int kType>
struct RowsIn {
    const typename Elem<kType>::T* logits;
    int64_t vocab, stride;
    int64_t span;
    int32_t nseg;
    float c, c_low;                              // log2(e) / T and what its rounding left

    __device__ __forceinline__ Segment<kType> segment(uint32_t block) const {
        constexpr int E = Elem<kType>::kE;
        const uint32_t row = block / (uint32_t)nseg, k = block % (uint32_t)nseg;
        const int64_t words = (vocab + E - 1) / E;
        Segment<kType> s;
        s.row = row;
        s.x = logits + (int64_t)row * stride;
        s.vocab = vocab;
        s.begin = (int64_t)k * span;
        s.end = s.begin + span < words ? s.begin + span : words;
        return s;
    }
};

// The part of a segment: each thread runs over its words with a maximum of its
// own, rescaling what it has when a chunk raises it; the threads join at the
// end.  Returned to every thread of wave 0.  kListed: `marks` has a bit set
// for each entry to leave out.  kTop: the threads' largest entry of each chunk
// goes to chunk_best, `mine` is its largest of all.
template <int kType, int kVecs, bool kListed, bool kTop>
__device__ __forceinline__ Part segment_part(const Segment<kType>& seg, float c,
                                             const uint32_t* marks, float* chunk_best, Part* red,
                                             float& mine) {
    constexpr int E = Elem<kType>::kE;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int n = seg.template chunks<kVecs>();
    float m = -INFINITY, s = 0.0f, u = 0.0f;
    for (int ch = 0; ch < n; ++ch) {
        u32x4 r[kVecs];
        seg.template load<kVecs>(ch, r);
        if (kListed) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int at = ((ch * kVecs + i) * kBlock + (int)threadIdx.x) * E;
                const uint32_t bits = (marks[at >> 5] >> (at & 31)) & ((1u << E) - 1);
                if (bits) {
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (bits >> e & 1) {
                            if (kType == FLASHOPT_FP32) r[i][e & 3] = Elem<kType>::kMinusInf;
                            else if (e & 1) r[i][e >> 1] = (r[i][e >> 1] & 0xFFFFu) | (Elem<kType>::kMinusInf & 0xFFFF0000u);
                            else r[i][e >> 1] = (r[i][e >> 1] & 0xFFFF0000u) | (Elem<kType>::kMinusInf & 0xFFFFu);
                        }
                }
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) top = fmaxf(top, Elem<kType>::get(r[i], e));
        if (kTop) chunk_best[ch * kBlock + threadIdx.x] = top;
        const float m_new = fmaxf(m, top);
        const float shift = m_new == -INFINITY ? 0.0f : m_new;    // nothing yet: every e_j is 0
        const float D = fmaxf((m - m_new) * c, -200.0f), f = exp2_hw(D);
        float cs = 0.0f, cu = 0.0f;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float d = (Elem<kType>::get(r[i], e) - shift) * c;
                const float p = exp2_hw(d);
                cs += p;
                // p is 0 below -150: the bound keeps 0 * -inf out of the sum
                if (!kListed) cu = __builtin_fmaf(p, fmaxf(d, -200.0f), cu);
            }
        if (!kListed) u = f * (u + D * s) + cu;
        s = s * f + cs;
        m = m_new;
    }
    mine = m;
    const float wm = wave_max(m);
    const float D = fmaxf((m - wm) * c, -200.0f), f = exp2_hw(D);
    // a lane of -inf alone has s = 0, one of NaN alone keeps it
    const float ws = wave_sum(s * f), wu = kListed ? 0.0f : wave_sum(f * (u + D * s));
    if (lane == 0) red[wave] = Part{wm, ws, wu, 0.0f};
    __syncthreads();
    Part p = {-INFINITY, 0.0f, 0.0f, 0.0f};
    if (wave == 0) p = join_parts(red, kWavesPerBlock, c);
    return p;
}

template <int kType, int kVecs, bool kTop, int kGrad>            // kGrad 1: of logprob, 2: and of entropy
__global__ __launch_bounds__(kBlock) void prob_kernel(RowsIn<kType> in, ProbOut out, int top,
                                                      Part* part, uint64_t* lists,
                                                      ProbGrad<kType> G) {
    extern __shared__ float chunk_best[];
    __shared__ Part red[kWavesPerBlock];
    __shared__ ProbStats shared_stats;
    const Segment<kType> seg = in.segment(blockIdx.x);
    float mine;
    const Part p = segment_part<kType, kVecs, false, kTop>(seg, in.c, nullptr, chunk_best, red, mine);
    if (in.nseg > 1) {
        if (threadIdx.x == 0) part[blockIdx.x] = p;
    } else if (threadIdx.x == 0) {
        const ProbStats st = prob_stats(p);
        shared_stats = st;
        write_prob<kType>(seg.x, seg.vocab, seg.row, in.c, st, out);
    }
    if (kTop) {
        __shared__ TopShared sh;
        if (in.nseg > 1) {
            uint64_t* list = lists + (int64_t)blockIdx.x * top;
            segment_top<kType, kVecs>(seg, chunk_best, mine, top, sh, [&](uint32_t k, uint64_t e) { list[k] = e; });
        } else {
            segment_top<kType, kVecs>(seg, chunk_best, mine, top, sh, [&](uint32_t k, uint64_t e) {
                write_top(out, seg.row, top, (int)k, e, in.c, shared_stats);
            });
        }
    }
    if (kGrad) {
        __syncthreads();
        prob_grad_segment<kType, kVecs, kGrad == 2>(seg, in.c, shared_stats, out.targets, G);
    }
}

template <int kType>
__global__ __launch_bounds__(kBlock) void prob_join_kernel(RowsIn<kType> in, int64_t rows,
                                                           ProbOut out, int top, const Part* part,
                                                           const uint64_t* lists) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t row = (int64_t)blockIdx.x * kWavesPerBlock + threadIdx.x / kWave;
    if (row >= rows) return;
    const ProbStats st = prob_stats(join_parts(part + row * in.nseg, in.nseg, in.c));
    if (lane == 0) write_prob<kType>(in.logits + row * in.stride, in.vocab, row, in.c, st, out);
    if (top > 0) {
        // lane b walks the list of segment b, best first (a row has at most 64)
        const uint64_t* mine = lists + (row * in.nseg + lane) * top;
        int at = 0;
        uint64_t head = lane < in.nseg ? mine[0] : 0;
        for (int k = 0; k < top; ++k) {
            const uint64_t best = wave_max_u64(head);
            if (head == best && lane < in.nseg) head = ++at < top ? mine[at] : 0;
            if (lane == 0) write_top(out, row, top, k, best, in.c, st);
        }
    }
}

template <int kType, int kVecs, bool kEntropy>
__global__ __launch_bounds__(kBlock) void prob_grad_kernel(RowsIn<kType> in, const int64_t* targets,
                                                           const ProbStats* stats,
                                                           ProbGrad<kType> G) {
    const Segment<kType> seg = in.segment(blockIdx.x);
    prob_grad_segment<kType, kVecs, kEntropy>(seg, in.c, stats[seg.row], targets, G);
}

template <int kType, int kVecs, bool kGrad>
__global__ __launch_bounds__(kBlock) void distill_kernel(RowsIn<kType> in, DistillIn list,
                                                         Part* part, float* loss,
                                                         DistillStats* stats,
                                                         DistillGrad<kType> G) {
    extern __shared__ uint32_t marks[];
    __shared__ Part red[kWavesPerBlock];
    __shared__ DistillStats shared_stats;
    const Segment<kType> seg = in.segment(blockIdx.x);
    const int words = seg.template chunks<kVecs>() * (kChunk<kType, kVecs> / 32);
    for (int i = threadIdx.x; i < words; i += kBlock) marks[i] = 0;
    __syncthreads();
    if (threadIdx.x < list.top) {
        const int64_t id = list.ids[seg.row * list.top + threadIdx.x];
        const int64_t at = id - seg.first_id();
        if (id >= seg.first_id() && id < seg.end_id()) atomicOr(&marks[at >> 5], 1u << (at & 31));
    }
    __syncthreads();
    float mine;
    const Part p = segment_part<kType, kVecs, true, false>(seg, in.c, marks, nullptr, red, mine);
    if (in.nseg > 1) {
        if (threadIdx.x == 0) part[blockIdx.x] = p;
    } else if (threadIdx.x < kWave) {
        float l;
        const DistillStats st = distill_stats<kType>(seg.x, seg.vocab, seg.row, in.c, in.c_low, list, p, l);
        if (threadIdx.x == 0) {
            if (loss) loss[seg.row] = l;
            stats[seg.row] = st;
            shared_stats = st;
        }
    }
    if (kGrad) {
        __syncthreads();
        distill_grad_segment<kType, kVecs>(seg, in.c, shared_stats, list, G);
    }
}

template <int kType>
__global__ __launch_bounds__(kBlock) void distill_join_kernel(RowsIn<kType> in, int64_t rows,
                                                              DistillIn list, const Part* part,
                                                              float* loss, DistillStats* stats) {
    const int64_t row = (int64_t)blockIdx.x * kWavesPerBlock + threadIdx.x / kWave;
    if (row >= rows) return;
    const Part rest = join_parts(part + row * in.nseg, in.nseg, in.c);
    float l;
    const DistillStats st = distill_stats<kType>(in.logits + row * in.stride, in.vocab, row, in.c,
                                                 in.c_low, list, rest, l);
    if ((threadIdx.x & (kWave - 1)) == 0) {
        if (loss) loss[row] = l;
        stats[row] = st;
    }
}

template <int kType, int kVecs>
__global__ __launch_bounds__(kBlock) void distill_grad_kernel(RowsIn<kType> in, DistillIn list,
                                                              const DistillStats* stats,
                                                              DistillGrad<kType> G) {
    const Segment<kType> seg = in.segment(blockIdx.x);
    distill_grad_segment<kType, kVecs>(seg, in.c, stats[seg.row], list, G);
}

// ---- host ---------------------------------------------------------------------

static int check_rows(const void* logits, int32_t type, int64_t rows, int64_t vocab, int64_t stride,
                      double temperature) {
    if (!valid_type(type)) return FLASHOPT_ERR_ARG;
    if (rows < 0 || vocab < 1 || vocab > FLASHOPT_VOCAB_MAX || stride < vocab ||
        stride > kMaxNumel || rows > INT32_MAX / ((vocab + 4095) / 4096))
        return FLASHOPT_ERR_SIZE;
    // 1/T and log2(e)/T are used as normal binary32 numbers
    if (!(temperature >= 0x1p-126) || !(temperature <= 0x1p126)) return FLASHOPT_ERR_ARG;
    if (rows == 0) return FLASHOPT_OK;
    if (!logits) return FLASHOPT_ERR_NULL;
    if (!aligned(logits, type_size(type))) return FLASHOPT_ERR_ALIGN;
    return FLASHOPT_OK;
}

static int check_grad(const void* grad, int32_t type, int64_t vocab, int64_t grad_stride) {
    if (!grad) return FLASHOPT_ERR_NULL;
    if (grad_stride < vocab || grad_stride > kMaxNumel) return FLASHOPT_ERR_SIZE;
    if (!aligned(grad, type_size(type))) return FLASHOPT_ERR_ALIGN;
    return FLASHOPT_OK;
}

static int check_workspace(const void* workspace, size_t have, size_t need) {
    if (need == 0) return FLASHOPT_OK;
    if (!workspace) return FLASHOPT_ERR_NULL;
    if (have < need || !aligned(workspace, 256)) return FLASHOPT_ERR_WORKSPACE;
    return FLASHOPT_OK;
}

static int check_list(const int64_t* top_id, const float* top_logprob, int32_t top, int64_t vocab) {
    if (top < 1 || top > FLASHOPT_TOP_MAX || top > vocab) return FLASHOPT_ERR_ARG;
    if (!top_id || !top_logprob) return FLASHOPT_ERR_NULL;
    if (!aligned(top_id, 8) || !aligned(top_logprob, 4)) return FLASHOPT_ERR_ALIGN;
    return FLASHOPT_OK;
}

// How a call cuts its rows.  A block streams a segment of a row; with many
// rows a segment is the whole row and nothing has to be joined, with fewer the
// rows are cut until about kBlocksWanted blocks run (at most kMaxSegments a row,
// which one wave joins), and with very few the chunks are the short ones.  A
// segment is at most kMaxChunks chunks, whose maxima or marks lie in LDS.
constexpr int64_t kBlocksWanted = 1024;
constexpr int64_t kMaxSegments = 64;
constexpr int kMaxChunks = 16;
struct Cut {
    int vecs;
    int64_t span;                                // 16-byte words of a segment
    int32_t nseg;
    int chunks;                                  // of a segment
};
static Cut cut_rows(int32_t type, int64_t rows, int64_t vocab) {
    const int64_t e = type == FLASHOPT_FP32 ? 4 : 8, words = (vocab + e - 1) / e;
    Cut k;
    const int64_t lng = (words + kLong * kBlock - 1) / (kLong * kBlock);
    k.vecs = rows * lng < 256 ? kShort : kLong;
    const int64_t step = (int64_t)k.vecs * kBlock, chunks = (words + step - 1) / step;
    int64_t want = (kBlocksWanted + rows - 1) / (rows < 1 ? 1 : rows);
    want = want < 1 ? 1 : want > kMaxSegments ? kMaxSegments : want;
    k.chunks = (int)((chunks + want - 1) / want);
    if (k.chunks > kMaxChunks) k.chunks = kMaxChunks;
    k.span = k.chunks * step;
    k.nseg = (int32_t)((words + k.span - 1) / k.span);
    return k;
}

// a row that one block holds needs no workspace
static size_t parts_bytes(const Cut& k, int64_t rows) {
    if (k.nseg == 1) return 0;
    const size_t b = (size_t)(rows * k.nseg) * sizeof(Part);
    return (b + 255) & ~size_t(255);
}

// f is called with the type and the chunk's words as compile-time constants
template <typename F>
static int by_type(int32_t type, int vecs, F f) {
    auto with = [&](auto t) {
        if (vecs == kLong) f(t, std::integral_constant<int, kLong>());
        else f(t, std::integral_constant<int, kShort>());
    };
    if (type == FLASHOPT_BF16) with(std::integral_constant<int, FLASHOPT_BF16>());
    else if (type == FLASHOPT_FP16) with(std::integral_constant<int, FLASHOPT_FP16>());
    else with(std::integral_constant<int, FLASHOPT_FP32>());
    return launch_status();
}

struct Rows {                                    // a call's logits
    const void* logits;
    int32_t type;
    int64_t rows, vocab, stride;
    double temperature;
};

template <int kType>
static RowsIn<kType> rows_in(const Rows& a, const Cut& k) {
    RowsIn<kType> in;
    in.logits = (const typename Elem<kType>::T*)a.logits;
    in.vocab = a.vocab;
    in.stride = a.stride;
    in.span = k.span;
    in.nseg = k.nseg;
    const double c = 1.4426950408889634073599 / a.temperature;
    in.c = (float)c;
    in.c_low = (float)(c - (double)in.c);
    return in;
}

static dim3 join_grid(int64_t rows) {
    return dim3((unsigned)((rows + kWavesPerBlock - 1) / kWavesPerBlock));
}

// The forward pass; with `grad`, rows that one block holds get their gradient
// in the same launch, others in one more.
static int launch_prob(const Rows& a, const ProbOut& out, int32_t top, void* workspace,
                       const float* grad_logprob, const float* grad_entropy, void* grad,
                       int64_t grad_stride, hipStream_t st) {
    const Cut k = cut_rows(a.type, a.rows, a.vocab);
    Part* part = (Part*)workspace;
    uint64_t* lists = (uint64_t*)((char*)workspace + parts_bytes(k, a.rows));
    return by_type(a.type, k.vecs, [&](auto t, auto v) {
        constexpr int kType = decltype(t)::value, kVecs = decltype(v)::value;
        const RowsIn<kType> in = rows_in<kType>(a, k);
        const dim3 grid((unsigned)(a.rows * k.nseg));
        const ProbGrad<kType> G = {grad_logprob, grad_entropy, (typename Elem<kType>::T*)grad,
                                   grad_stride, (float)(1.0 / a.temperature)};
        const size_t lds = top > 0 ? (size_t)k.chunks * kBlock * sizeof(float) : 0;
        if (top > 0)
            hipLaunchKernelGGL((prob_kernel<kType, kVecs, true, 0>), grid, dim3(kBlock), lds, st, in,
                               out, top, part, lists, G);
        else if (!grad || k.nseg > 1)
            hipLaunchKernelGGL((prob_kernel<kType, kVecs, false, 0>), grid, dim3(kBlock), 0, st, in,
                               out, 0, part, lists, G);
        else if (grad_entropy)
            hipLaunchKernelGGL((prob_kernel<kType, kVecs, false, 2>), grid, dim3(kBlock), 0, st, in,
                               out, 0, part, lists, G);
        else
            hipLaunchKernelGGL((prob_kernel<kType, kVecs, false, 1>), grid, dim3(kBlock), 0, st, in,
                               out, 0, part, lists, G);
        if (k.nseg > 1)
            hipLaunchKernelGGL((prob_join_kernel<kType>), join_grid(a.rows), dim3(kBlock), 0, st, in,
                               a.rows, out, top, part, lists);
    });
}

static int launch_prob_grad(const Rows& a, const int64_t* targets, const float* stats,
                            const float* grad_logprob, const float* grad_entropy, void* grad,
                            int64_t grad_stride, hipStream_t st) {
    Cut k = cut_rows(a.type, a.rows, a.vocab);
    return by_type(a.type, k.vecs, [&](auto t, auto v) {
        constexpr int kType = decltype(t)::value, kVecs = decltype(v)::value;
        const RowsIn<kType> in = rows_in<kType>(a, k);
        const dim3 grid((unsigned)(a.rows * k.nseg));
        const ProbGrad<kType> G = {grad_logprob, grad_entropy, (typename Elem<kType>::T*)grad,
                                   grad_stride, (float)(1.0 / a.temperature)};
        if (grad_entropy)
            hipLaunchKernelGGL((prob_grad_kernel<kType, kVecs, true>), grid, dim3(kBlock), 0, st, in,
                               targets, (const ProbStats*)stats, G);
        else
            hipLaunchKernelGGL((prob_grad_kernel<kType, kVecs, false>), grid, dim3(kBlock), 0, st, in,
                               targets, (const ProbStats*)stats, G);
    });
}

static int launch_distill(const Rows& a, const DistillIn& list, void* workspace, float* loss,
                          float* stats, const float* grad_loss, void* grad, int64_t grad_stride,
                          hipStream_t st) {
    const Cut k = cut_rows(a.type, a.rows, a.vocab);
    Part* part = (Part*)workspace;
    return by_type(a.type, k.vecs, [&](auto t, auto v) {
        constexpr int kType = decltype(t)::value, kVecs = decltype(v)::value;
        const RowsIn<kType> in = rows_in<kType>(a, k);
        const dim3 grid((unsigned)(a.rows * k.nseg));
        const DistillGrad<kType> G = {grad_loss, (typename Elem<kType>::T*)grad, grad_stride,
                                      (float)(1.0 / a.temperature)};
        const size_t lds = (size_t)k.chunks * kChunk<kType, kVecs> / 8;
        if (grad && k.nseg == 1)
            hipLaunchKernelGGL((distill_kernel<kType, kVecs, true>), grid, dim3(kBlock), lds, st, in,
                               list, part, loss, (DistillStats*)stats, G);
        else
            hipLaunchKernelGGL((distill_kernel<kType, kVecs, false>), grid, dim3(kBlock), lds, st, in,
                               list, part, loss, (DistillStats*)stats, G);
        if (k.nseg > 1) {
            hipLaunchKernelGGL((distill_join_kernel<kType>), join_grid(a.rows), dim3(kBlock), 0, st,
                               in, a.rows, list, part, loss, (DistillStats*)stats);
            if (grad)
                hipLaunchKernelGGL((distill_grad_kernel<kType, kVecs>), grid, dim3(kBlock), 0, st, in,
                                   list, (const DistillStats*)stats, G);
        }
    });
}

static int launch_distill_grad(const Rows& a, const DistillIn& list, const float* stats,
                               const float* grad_loss, void* grad, int64_t grad_stride,
                               hipStream_t st) {
    const Cut k = cut_rows(a.type, a.rows, a.vocab);
    return by_type(a.type, k.vecs, [&](auto t, auto v) {
        constexpr int kType = decltype(t)::value, kVecs = decltype(v)::value;
        const DistillGrad<kType> G = {grad_loss, (typename Elem<kType>::T*)grad, grad_stride,
                                      (float)(1.0 / a.temperature)};
        hipLaunchKernelGGL((distill_grad_kernel<kType, kVecs>), dim3((unsigned)(a.rows * k.nseg)),
                           dim3(kBlock), 0, st, rows_in<kType>(a, k), list,
                           (const DistillStats*)stats, G);
    });
}

}  // namespace flashopt

using namespace flashopt;

extern "C" {

size_t flashopt_logprob_workspace_bytes(int32_t type, int64_t rows, int64_t vocab, int32_t top) {
    if (!valid_type(type) || rows < 0 || vocab < 1 || vocab > FLASHOPT_VOCAB_MAX || top < 0 ||
        top > FLASHOPT_TOP_MAX || rows > INT32_MAX / ((vocab + 4095) / 4096))
        return 0;
    const Cut k = cut_rows(type, rows, vocab);
    if (k.nseg == 1) return 0;
    return parts_bytes(k, rows) + (size_t)(rows * k.nseg) * (size_t)top * sizeof(uint64_t);
}

int flashopt_logprob(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                     int64_t stride, double temperature, const int64_t* targets, int32_t top,
                     void* workspace, size_t workspace_bytes, float* logprob, float* entropy,
                     float* stats, float* top_logprob, int64_t* top_id, void* stream) {
    const int e = check_rows(logits, type, rows, vocab, stride, temperature);
    if (e) return e;
    if (top < 0 || top > FLASHOPT_TOP_MAX || top > vocab) return FLASHOPT_ERR_ARG;
    if (rows == 0) return FLASHOPT_OK;
    if ((top > 0 && (!top_logprob || !top_id)) || (logprob && !targets)) return FLASHOPT_ERR_NULL;
    if (!aligned(targets, 8) || !aligned(logprob, 4) || !aligned(entropy, 4) ||
        !aligned(stats, 16) || !aligned(top_logprob, 4) || !aligned(top_id, 8))
        return FLASHOPT_ERR_ALIGN;
    const int w = check_workspace(workspace, workspace_bytes,
                                  flashopt_logprob_workspace_bytes(type, rows, vocab, top));
    if (w) return w;
    return launch_prob({logits, type, rows, vocab, stride, temperature},
                       {targets, logprob, entropy, (ProbStats*)stats, top_logprob, top_id}, top,
                       workspace, nullptr, nullptr, nullptr, 0, (hipStream_t)stream);
}

int flashopt_logprob_backward(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                              int64_t stride, double temperature, const int64_t* targets,
                              const float* stats, const float* grad_logprob,
                              const float* grad_entropy, void* grad, int64_t grad_stride,
                              void* stream) {
    const int e = check_rows(logits, type, rows, vocab, stride, temperature);
    if (e) return e;
    if (rows == 0) return FLASHOPT_OK;
    if (!stats || (grad_logprob && !targets)) return FLASHOPT_ERR_NULL;
    if (!aligned(stats, 16) || !aligned(targets, 8) || !aligned(grad_logprob, 4) ||
        !aligned(grad_entropy, 4))
        return FLASHOPT_ERR_ALIGN;
    const int g = check_grad(grad, type, vocab, grad_stride);
    if (g) return g;
    return launch_prob_grad({logits, type, rows, vocab, stride, temperature}, targets, stats,
                            grad_logprob, grad_entropy, grad, grad_stride, (hipStream_t)stream);
}

int flashopt_logprob_grad(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                          int64_t stride, double temperature, const int64_t* targets,
                          const float* grad_logprob, const float* grad_entropy, void* workspace,
                          size_t workspace_bytes, float* logprob, float* entropy, float* stats,
                          void* grad, int64_t grad_stride, void* stream) {
    const int e = check_rows(logits, type, rows, vocab, stride, temperature);
    if (e) return e;
    if (rows == 0) return FLASHOPT_OK;
    if (!stats || ((logprob || grad_logprob) && !targets)) return FLASHOPT_ERR_NULL;
    if (!aligned(targets, 8) || !aligned(logprob, 4) || !aligned(entropy, 4) ||
        !aligned(stats, 16) || !aligned(grad_logprob, 4) || !aligned(grad_entropy, 4))
        return FLASHOPT_ERR_ALIGN;
    const int g = check_grad(grad, type, vocab, grad_stride);
    if (g) return g;
    const int w = check_workspace(workspace, workspace_bytes,
                                  flashopt_logprob_workspace_bytes(type, rows, vocab, 0));
    if (w) return w;
    const Rows a = {logits, type, rows, vocab, stride, temperature};
    const int f = launch_prob(a, {targets, logprob, entropy, (ProbStats*)stats, nullptr, nullptr}, 0,
                              workspace, grad_logprob, grad_entropy, grad, grad_stride,
                              (hipStream_t)stream);
    if (f || cut_rows(type, rows, vocab).nseg == 1) return f;
    return launch_prob_grad(a, targets, stats, grad_logprob, grad_entropy, grad, grad_stride,
                            (hipStream_t)stream);
}

size_t flashopt_distill_workspace_bytes(int32_t type, int64_t rows, int64_t vocab) {
    return flashopt_logprob_workspace_bytes(type, rows, vocab, 0);
}

int flashopt_distill(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                     int64_t stride, double temperature, const int64_t* top_id,
                     const float* top_logprob, int32_t top, int32_t tail, void* workspace,
                     size_t workspace_bytes, float* loss, float* stats, void* stream) {
    const int e = check_rows(logits, type, rows, vocab, stride, temperature);
    if (e) return e;
    if (top < 1 || top > FLASHOPT_TOP_MAX || top > vocab || tail < 0 || tail > 1)
        return FLASHOPT_ERR_ARG;
    if (rows == 0) return FLASHOPT_OK;
    const int l = check_list(top_id, top_logprob, top, vocab);
    if (l) return l;
    if (!stats) return FLASHOPT_ERR_NULL;
    if (!aligned(stats, 16) || !aligned(loss, 4)) return FLASHOPT_ERR_ALIGN;
    const int w = check_workspace(workspace, workspace_bytes,
                                  flashopt_distill_workspace_bytes(type, rows, vocab));
    if (w) return w;
    return launch_distill({logits, type, rows, vocab, stride, temperature},
                          {top_id, top_logprob, top, tail}, workspace, loss, stats, nullptr, nullptr,
                          0, (hipStream_t)stream);
}

int flashopt_distill_backward(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                              int64_t stride, double temperature, const int64_t* top_id,
                              const float* top_logprob, int32_t top, const float* stats,
                              const float* grad_loss, void* grad, int64_t grad_stride,
                              void* stream) {
    const int e = check_rows(logits, type, rows, vocab, stride, temperature);
    if (e) return e;
    if (top < 1 || top > FLASHOPT_TOP_MAX || top > vocab) return FLASHOPT_ERR_ARG;
    if (rows == 0) return FLASHOPT_OK;
    const int l = check_list(top_id, top_logprob, top, vocab);
    if (l) return l;
    if (!stats || !grad_loss) return FLASHOPT_ERR_NULL;
    if (!aligned(stats, 16) || !aligned(grad_loss, 4)) return FLASHOPT_ERR_ALIGN;
    const int g = check_grad(grad, type, vocab, grad_stride);
    if (g) return g;
    return launch_distill_grad({logits, type, rows, vocab, stride, temperature},
                               {top_id, top_logprob, top, 0}, stats, grad_loss, grad, grad_stride,
                               (hipStream_t)stream);
}

int flashopt_distill_grad(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                          int64_t stride, double temperature, const int64_t* top_id,
                          const float* top_logprob, int32_t top, int32_t tail,
                          const float* grad_loss, void* workspace, size_t workspace_bytes,
                          float* loss, float* stats, void* grad, int64_t grad_stride,
                          void* stream) {
    const int e = check_rows(logits, type, rows, vocab, stride, temperature);
    if (e) return e;
    if (top < 1 || top > FLASHOPT_TOP_MAX || top > vocab || tail < 0 || tail > 1)
        return FLASHOPT_ERR_ARG;
    if (rows == 0) return FLASHOPT_OK;
    const int l = check_list(top_id, top_logprob, top, vocab);
    if (l) return l;
    if (!stats || !grad_loss) return FLASHOPT_ERR_NULL;
    if (!aligned(stats, 16) || !aligned(loss, 4) || !aligned(grad_loss, 4))
        return FLASHOPT_ERR_ALIGN;
    const int g = check_grad(grad, type, vocab, grad_stride);
    if (g) return g;
    const int w = check_workspace(workspace, workspace_bytes,
                                  flashopt_distill_workspace_bytes(type, rows, vocab));
    if (w) return w;
    return launch_distill({logits, type, rows, vocab, stride, temperature},
                          {top_id, top_logprob, top, tail}, workspace, loss, stats, grad_loss, grad,
                          grad_stride, (hipStream_t)stream);
}

}  // extern "C"
