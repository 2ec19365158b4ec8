// Rows of logits (include/flashopt_lm.h): log probabilities of given tokens
// with entropy and top alternatives, distillation from a teacher's top
// logits, and their gradients.
//
// Mathematics.  With c = log2(e) / T and m the row's largest entry, its
// distribution is p_j = 2^((x_j - m) c) / S, S = sum_j 2^((x_j - m) c).  A thread
// sums, over its words of a segment of a row, relative to its own largest entry,
//   S = sum_j e_j,  U = sum_j e_j d_j   (d_j = (x_j - m) c, e_j = 2^d_j);
// joining chunks, threads, waves and segments rescales them to the larger one's:
//   S = sum S_k 2^(D_k),  U = sum 2^(D_k) (U_k + D_k S_k),  D_k = (m_k - m) c <= 0.
// Then log2 p_j = d_j - log2 S and H = ln2 (log2 S - U / S).  With m the largest
// entry S is at least 1 and U at most 0: no sum cancels, and where one token is
// nearly certain all of log2 S, U / S and its d are as small as the result.  (A
// shift that lies k bits lower leaves differences of numbers near k there.)
//
// The gradients are elementwise in the row's numbers: one more pass over the
// words, plus a few entries (the given token, the teacher's alternatives) that
// the block writes again after its dense pass, from logits it read before it, so
// that a gradient may replace its logits.
//
// Rows of BF16 bring 10.5 issue slots an entry (half for the maximum, of packed
// pairs; unpack, subtract, multiply, exp2 at a quarter of the rate, bound, two
// sums) for 2 bytes: 80 us at 2048 x 128256 where HBM takes 97, so the forward pass
// is bound by HBM with some blocks a CU (2048 x 128256 BF16: 98 us, 5.4 TB/s; with
// the 64 best entries 125) and by the sums with one (300 x 131072: 24).
#include <cmath>

#include "logits.hpp"

namespace flashopt {

// 16-byte words of a chunk per thread: 8 streams best; with few rows 2 give
// more, shorter work items.
constexpr int kLong = 8, kShort = 2;
constexpr int kMaxSegments = 64;                 // of a row: one wave joins them
template <int kType, int kVecs> constexpr int kChunk = kVecs * kBlock * Elem<kType>::kE;

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

__device__ __forceinline__ void write_top(const ProbOut& o, int64_t row, int top, int k,
                                          uint64_t e, float c, const ProbStats& st) {
    o.top_id[row * top + k] = entry_id(e);
    o.top_logprob[row * top + k] = ((key_value(entry_key(e)) - st.m) * c - st.l2s) * kLn2;
}

// A segment of a row: the words [begin, end) of 16 bytes; the row's last
// word may be partial.  Chunks are kVecs words of each of kThreads threads.
template <int kType, int kThreads = kBlock>
struct Segment {
    typedef typename Elem<kType>::T T;
    const T* x;
    int64_t vocab, begin, end;                   // words
    int64_t row;

    // kLast: nothing reads these logits after this call's gradient.  With the
    // non-temporal hint here and on the gradient's stores, the rows that other
    // blocks have read once stay in the last-level cache until their gradient:
    // 4096 x 128256 BF16 distillation takes 500 us, 646 without either hint.
    template <int kVecs, bool kLast = false>
    __device__ __forceinline__ void load(int64_t chunk, u32x4* r) const {
        const int64_t v0 = begin + chunk * (kVecs * kThreads);
        if (whole<kVecs>(v0)) {                  // all loads in flight at once
            const T* p = x + v0 * Elem<kType>::kE;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const auto* w = reinterpret_cast<const u32x4_any*>(
                    p + (threadIdx.x + i * kThreads) * Elem<kType>::kE);
                r[i] = kLast ? __builtin_nontemporal_load(w) : *w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int64_t w = v0 + threadIdx.x + i * kThreads;
                // words past the segment belong to another block, or to no row
                r[i] = load_vec<kType>(x, w, w < end ? vocab : 0, Elem<kType>::kMinusInf);
            }
        }
    }
    // words from the i-th on are past the segment (equal for the block's threads)
    template <int kVecs>
    __device__ __forceinline__ bool none(int64_t chunk, int i) const {
        return begin + chunk * (kVecs * kThreads) + i * kThreads >= end;
    }
    // a chunk of whole words, all of the segment (equal for the block's threads)
    template <int kVecs>
    __device__ __forceinline__ bool whole(int64_t v0) const {
        const int64_t e = v0 + kVecs * kThreads;
        return e <= end && e * Elem<kType>::kE <= vocab;
    }
    template <int kVecs>
    __device__ __forceinline__ void store(T* g, int64_t chunk, int i, u32x4 o) const {
        const int64_t v0 = begin + chunk * (kVecs * kThreads);
        if (whole<kVecs>(v0)) {
            __builtin_nontemporal_store(
                o, reinterpret_cast<u32x4_any*>(g + v0 * Elem<kType>::kE +
                                                (threadIdx.x + i * kThreads) * Elem<kType>::kE));
        } else {
            const int64_t w = v0 + threadIdx.x + i * kThreads;
            store_vec<kType>(g, w, w < end ? vocab : 0, o);
        }
    }
    template <int kVecs>
    __device__ __forceinline__ int chunks() const {
        return (int)((end - begin + kVecs * kThreads - 1) / (kVecs * kThreads));
    }
    __device__ __forceinline__ int64_t first_id() const { return begin * Elem<kType>::kE; }
    __device__ __forceinline__ int64_t end_id() const {
        const int64_t e = end * Elem<kType>::kE;
        return e < vocab ? e : vocab;
    }
};

// ---- the best entries of a segment ----------------------------------------------

constexpr int kFound = 512;                      // candidates kept before the exact search is taken

constexpr int kPairs = 1024;                     // 63 threads with all of a segment's chunks and more

struct TopShared {
    float best[kBlock];                          // each thread's largest entry
    uint16_t pair[kPairs];                       // chunk * kBlock + thread
    uint64_t found[kFound];
    uint32_t npair, nfound, count[2][kWavesPerBlock];
};

// The `need` best entries into found[0, need), whatever the values: an entry
// is its value and id as one number, so all differ, and the bits of the
// need-th largest are set from the highest down, counting the entries at or
// above each trial.  One pass over the segment a bit: the path of rows with
// hundreds of equal entries at the border or with NaN.
template <int kType>
__device__ __noinline__ void search_top(const Segment<kType>& seg, uint32_t need, TopShared& sh) {
    constexpr int E = Elem<kType>::kE;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    auto each = [&](auto f) {
        for (int64_t w = seg.begin + threadIdx.x; w < seg.end; w += kBlock) {
            const u32x4 r = load_vec<kType>(seg.x, w, seg.vocab, Elem<kType>::kMinusInf);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (w * E + e < seg.vocab) f(entry(Elem<kType>::get(r, e), (uint32_t)(w * E + e)));
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
        n = wave_reduce(n, 0u, [](uint32_t a, uint32_t b) { return a + b; });
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
// -256 ln(1 - top/256) of them, 74 for 64, are at or above it.  Only the words
// of a thread's chunk whose maximum is at or above it are read again: such
// pairs of thread and chunk are listed, and kVecs threads each take a pair.
template <int kType, int kVecs, typename Out>
__device__ __forceinline__ void segment_top(const Segment<kType>& seg, const float* chunk_best,
                                            float mine, int top, TopShared& sh, Out out) {
    constexpr int E = Elem<kType>::kE;
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t entries = seg.end_id() - seg.first_id();
    const uint32_t need = entries < top ? (uint32_t)entries : (uint32_t)top;
    sh.best[threadIdx.x] = mine;
    if (threadIdx.x == 0) sh.nfound = sh.npair = 0;
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
            const uint32_t at = atomicAdd(&sh.npair, 1u);
            if (at < (uint32_t)kPairs) sh.pair[at] = (uint16_t)(ch * kBlock + threadIdx.x);
        }
    }
    __syncthreads();
    const uint32_t npair = sh.npair;
    if (npair <= (uint32_t)kPairs)
        for (uint32_t p = threadIdx.x / kVecs; p < npair; p += kBlock / kVecs) {
            const int at = sh.pair[p], ch = at / kBlock, t = at % kBlock;
            const int64_t w = seg.begin + ((int64_t)ch * kVecs + threadIdx.x % kVecs) * kBlock + t;
            // a word past the segment is another block's
            const u32x4 r = load_vec<kType>(seg.x, w, w < seg.end ? seg.vocab : 0, Elem<kType>::kMinusInf);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float x = Elem<kType>::get(r, e);
                if (few ? x > low : x >= low) {              // padding is -inf, never taken
                    const uint32_t k = atomicAdd(&sh.nfound, 1u);
                    if (k < (uint32_t)kFound) sh.found[k] = entry(x, (uint32_t)(w * E + e));
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
    if (n < need || n > (uint32_t)kFound || npair > (uint32_t)kPairs) {      // equal for all threads
        search_top<kType>(seg, need, sh);
        n = need;
    }
    for (uint32_t t = threadIdx.x; t < n; t += kBlock) {
        const uint64_t x = sh.found[t];
        uint32_t rank = 0;
#pragma unroll 4
        for (uint32_t j = 0; j < n; ++j) rank += sh.found[j] > x ? 1u : 0u;
        if (rank < need) out(rank, x);
    }
    if (threadIdx.x >= need && threadIdx.x < (uint32_t)top) out(threadIdx.x, uint64_t(0));
}

// ---- sums ---------------------------------------------------------------------------

// S and U of N words relative to m, S by pairs: a sum that holds the 1 of the
// row's largest entry loses up to 2^-24 with each small one added to it.
template <int kType, bool kU, int N>
__device__ __forceinline__ void word_sums(const u32x4* r, float m, float c, float& s, float& u) {
    constexpr int E = Elem<kType>::kE;
    PairSum words;
    u = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        PairSum word;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float d = (Elem<kType>::get(r[i], e) - m) * c, p = exp2_hw(d);
            word.add(e, p);
            // where p is 0 the bound keeps 0 * -inf out of the sum
            if (kU) u = __builtin_fmaf(p, fmaxf(d, -200.0f), u);
        }
        words.add(i, word.total(E));
        __builtin_amdgcn_sched_barrier(0);       // a word's values at a time in registers
    }
    s = words.total(N);
}

// A thread's running sums of its words, relative to the largest of its entries
// so far.  The maximum of a chunk's words comes first: against a shift that earlier
// words fixed, raised when later ones exceed it, this costs 1.3 times the issue
// slots and no registers (2048 x 128256 BF16 98 us for 98, 300 x 131072 24 for 21).
template <int kType, bool kU>
struct Sums {
    float m, s, u, c;
    __device__ __forceinline__ explicit Sums(float c_)
        : m(-INFINITY), s(0.0f), u(0.0f), c(c_) {}

    // N words; returns their maximum
    template <int N>
    __device__ __forceinline__ float add(const u32x4* r) {
        const float top = largest<kType, N>(r);
        const float m_new = fmaxf(m, top);
        // -inf: nothing yet, every p is 0
        const float base = m_new == -INFINITY ? 0.0f : m_new;
        float cs, cu;
        word_sums<kType, kU, N>(r, base, c, cs, cu);
        const float D = fmaxf((m - m_new) * c, -200.0f), f = exp2_hw(D);
        if (kU) u = f * (u + D * s) + cu;
        s = s * f + cs;
        m = m_new;
        return top;
    }
};

// ---- gradients ------------------------------------------------------------------------

// 2^((x - m) c - a) for many x: one fma and one exp2 where m c is small
// enough, (x - m) formed first where it is not (beyond 2^20 the rounding of
// m c, at most 2^-24 of it, would no longer be small as an exponent; entries
// of the type's lowest value are there too).  What k = RN(m c + a) rounds away
// is the same for all x: `left` = m c + a - k, to be taken off the exponent.
struct Shift {
    float m, c, a, k, left;
    bool fast;
    __device__ __forceinline__ Shift(float m_, float c_, float a_) : m(m_), c(c_), a(a_) {
        const float hi = m * c, lo = __builtin_fmaf(m, c, -hi);
        k = hi + a;
        const float b = k - hi;
        left = lo + ((hi - (k - b)) + (a - b));
        fast = __builtin_fabsf(hi) < 0x1p20f;
    }
    template <bool kFast> __device__ __forceinline__ float exponent(float x) const {
        return kFast ? __builtin_fmaf(x, c, -k) : (x - m) * c - a;
    }
};

// grad_j = scale p_j (A + B d_j) with d_j = log2 p_j; given_grad at the given
// token.  1 / T is the scale, so that A and B do not overflow where the gradient
// does not; without the entropy it is part of A.
template <int kType>
struct ProbGrad {
    const float *grad_logprob, *grad_entropy;    // either may be null
    typename Elem<kType>::T* grad;
    int64_t stride;
    float inv_t;
};
template <bool kEntropy>
struct ProbCoef {
    Shift h;
    float A, B, gl, gh, scale, low;
    __device__ __forceinline__ ProbCoef(const ProbStats& st, float c, float gl_, float gh_, float inv_t)
        : h(st.m, c, st.l2s), gl(kEntropy ? gl_ : gl_ * inv_t),
          gh(st.on == 0.0f ? 0.0f : gh_), scale(inv_t) {         // whatever the upstream gradient
        A = -gl - gh * st.entropy;
        B = -gh * kLn2;
        low = -200.0f;
        if (h.fast) {                            // the exponent's constant part into the factors
            const float g = exp2_hw(-h.left);
            A = g * (A - B * h.left);
            B = g * B;
        }
    }
    template <bool kFast> __device__ __forceinline__ float value(float x) const {
        const float d = h.exponent<kFast>(x), p = exp2_hw(d);
        return kEntropy ? p * __builtin_fmaf(B, fmaxf(d, low), A) * scale : p * A;
    }
    __device__ __forceinline__ float at_given(float x, const ProbStats& st) const {
        const float v = given_grad<kEntropy>(x, st, h.c, gl, gh);
        return kEntropy ? v * scale : v;
    }
};
template <int kType, bool kEntropy>
__device__ __forceinline__ ProbCoef<kEntropy> prob_coef(const ProbStats& st, float c,
                                                        const ProbGrad<kType>& G, int64_t row,
                                                        bool given) {
    const float gl = given && st.on != 0.0f && G.grad_logprob ? G.grad_logprob[row] : 0.0f;
    return ProbCoef<kEntropy>(st, c, gl, kEntropy ? G.grad_entropy[row] : 0.0f, G.inv_t);
}

template <int kType>
struct DistillGrad {
    const float* grad_loss;
    typename Elem<kType>::T* grad;
    int64_t stride;
    float inv_t;
};

// the unlisted entries' gradient a e_j
struct RestCoef {
    Shift h;
    float a;
    __device__ __forceinline__ RestCoef(const DistillStats& st, float c, float w)
        : h(st.rest_m, c, st.rest_l2), a(w * st.coef) {
        if (h.fast) a *= exp2_hw(-h.left);
    }
    template <bool kFast> __device__ __forceinline__ float value(float x) const {
        return a * exp2_hw(h.exponent<kFast>(x));
    }
};

template <int kType, int kVecs, bool kFast, int kThreads, typename Coef>
__device__ __forceinline__ void grad_words(const Segment<kType, kThreads>& seg, const Coef& k,
                                           typename Elem<kType>::T* g) {
    constexpr int E = Elem<kType>::kE;
    const int n = seg.template chunks<kVecs>();
    for (int ch = 0; ch < n; ++ch) {
        u32x4 r[kVecs];
        seg.template load<kVecs, true>(ch, r);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            if (seg.template none<kVecs>(ch, i)) break;          // 501 x 50257 FP16: 37.1 us for 38.2
            float o[E];
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = k.template value<kFast>(Elem<kType>::get(r[i], e));
            seg.template store<kVecs>(g, ch, i, pack<kType>(o));
        }
    }
}
template <int kType, int kVecs, typename Coef>
__device__ __forceinline__ void grad_segment(const Segment<kType>& seg, const Coef& k,
                                             typename Elem<kType>::T* g) {
    __syncthreads();             // the given or listed entries were read before they are replaced
    if (k.h.fast) grad_words<kType, kVecs, true>(seg, k, g);
    else grad_words<kType, kVecs, false>(seg, k, g);
    __syncthreads();             // those entries' own gradients are written after the dense ones
}

template <int kType, int kVecs, bool kEntropy>
__device__ __forceinline__ void prob_grad_segment(const Segment<kType>& seg, float c,
                                                  const ProbStats& st, const Given& t,
                                                  const ProbGrad<kType>& G) {
    typename Elem<kType>::T* g = G.grad + seg.row * G.stride;
    const auto k = prob_coef<kType, kEntropy>(st, c, G, seg.row, t.id >= 0);
    grad_segment<kType, kVecs>(seg, k, g);
    if (threadIdx.x == 0 && t.id >= seg.first_id() && t.id < seg.end_id())
        g[t.id] = Elem<kType>::down(k.at_given(t.x, st));
}

template <int kType, int kVecs>
__device__ __forceinline__ void distill_grad_segment(const Segment<kType>& seg, float c,
                                                     const DistillStats& st, int top,
                                                     const Listed& l, const DistillGrad<kType>& G) {
    typename Elem<kType>::T* g = G.grad + seg.row * G.stride;
    const float w = st.on != 0.0f ? G.grad_loss[seg.row] * G.inv_t : 0.0f;
    grad_segment<kType, kVecs>(seg, RestCoef(st, c, w), g);
    if (threadIdx.x < kWave) {
        const float v = listed_grad(l, st, top, c, w);
        if (l.id >= seg.first_id() && l.id < seg.end_id()) g[l.id] = Elem<kType>::down(v);
    }
}

// ---- kernels: segments ------------------------------------------------------------------

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

// Entries marked in a bitmap become -inf; `at` is the word's first entry there.
template <int kType>
__device__ __forceinline__ void leave_out(u32x4& r, const uint32_t* marks, int at) {
    constexpr int E = Elem<kType>::kE;
    const uint32_t bits = (marks[at >> 5] >> (at & 31)) & ((1u << E) - 1);
    if (!bits) return;
    constexpr uint32_t kInf = Elem<kType>::kMinusInf;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t mask;
        if (kType == FLASHOPT_FP32) {
            mask = 0u - (bits >> i & 1u);
        } else {
            mask = ((0u - (bits >> (2 * i) & 1u)) & 0xFFFFu) | ((0u - (bits >> (2 * i + 1) & 1u)) << 16);
        }
        r[i] = (r[i] & ~mask) | (kInf & mask);
    }
}

// The part of a segment: each thread runs over its words, relative to its largest
// entry so far, and the threads join at the end.  Every wave gets it.  kListed:
// `marks` has a bit set for each entry to leave out.  kTop: the threads' largest
// entry of each chunk goes to chunk_best, `mine` is its largest of all.
template <int kType, int kVecs, bool kListed, bool kTop, int kThreads>
__device__ __forceinline__ Part segment_part(const Segment<kType, kThreads>& seg, float c,
                                             const uint32_t* marks, float* chunk_best, Part* red,
                                             float& mine) {
    const int n = seg.template chunks<kVecs>();
    Sums<kType, !kListed> sums(c);
    mine = -INFINITY;
    for (int ch = 0; ch < n; ++ch) {
        u32x4 r[kVecs];
        seg.template load<kVecs>(ch, r);
        if (kListed)
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                leave_out<kType>(r[i], marks, ((ch * kVecs + i) * kThreads + (int)threadIdx.x) * Elem<kType>::kE);
        // A last chunk that is not half full: two words at a time, those there are
        // (1000 x 50257 BF16: 25.4 us for 27.8; 4000 x 14000, 7/8 full: 26.0 for 26.0).
        float top = -INFINITY;
        if (kVecs == kShort || !seg.template none<kVecs>(ch, kVecs / 2)) {
            top = sums.template add<kVecs>(r);
        } else {
#pragma unroll
            for (int i = 0; i < kVecs; i += 2)
                if (!seg.template none<kVecs>(ch, i)) top = fmaxf(top, sums.template add<2>(r + i));
        }
        if (kTop) {
            chunk_best[ch * kThreads + threadIdx.x] = top;
            mine = fmaxf(mine, top);
        }
    }
    const Part p = wave_part<!kListed>(sums.m, sums.s, sums.u, c);
    if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = p;
    __syncthreads();
    return join_parts(red, kThreads / kWave, c);
}

template <int kType, int kVecs, bool kTop, int kGrad>            // kGrad 1: of logprob, 2: and of entropy
__global__ __launch_bounds__(kBlock) void prob_kernel(RowsIn<kType> in, ProbOut out, int top,
                                                      Part* part, uint64_t* lists,
                                                      ProbGrad<kType> G) {
    extern __shared__ float chunk_best[];
    __shared__ Part red[kWavesPerBlock];
    const Segment<kType> seg = in.segment(blockIdx.x);
    float mine;
    const Part p = segment_part<kType, kVecs, false, kTop>(seg, in.c, nullptr, chunk_best, red, mine);
    const ProbStats st = prob_stats(p);
    if (in.nseg > 1) {
        if (threadIdx.x == 0) part[blockIdx.x] = p;
    } else if (!kGrad && threadIdx.x == 0) {
        write_prob(seg.row, in.c, st, given_token<kType>(seg.x, seg.vocab, seg.row, out.targets), out);
    }
    if (kTop) {
        __shared__ TopShared sh;
        if (in.nseg > 1) {
            uint64_t* list = lists + (int64_t)blockIdx.x * top;
            segment_top<kType, kVecs>(seg, chunk_best, mine, top, sh, [&](uint32_t k, uint64_t e) { list[k] = e; });
        } else {
            segment_top<kType, kVecs>(seg, chunk_best, mine, top, sh, [&](uint32_t k, uint64_t e) {
                write_top(out, seg.row, top, (int)k, e, in.c, st);
            });
        }
    }
    if (kGrad) {
        const Given t = given_token<kType>(seg.x, seg.vocab, seg.row, out.targets);
        if (threadIdx.x == 0) write_prob(seg.row, in.c, st, t, out);
        prob_grad_segment<kType, kVecs, kGrad == 2>(seg, in.c, st, t, G);
    }
}

// The rows of several segments joined, one block of one wave a row.  Of the
// segments' lists, best first, the entries at or above a bound are ranked against
// each other: with r = ceil(top / nseg), the ceil(top / r)-th largest of the
// lists' r-th entries has that many times r entries at or above it.  If they are
// too many (equal ones), the lists are walked from their heads instead.
template <int kType>
__global__ __launch_bounds__(kWave) void prob_join_kernel(RowsIn<kType> in, ProbOut out, int top,
                                                          const Part* part,
                                                          const uint64_t* lists) {
    constexpr int kMost = 256;
    __shared__ uint64_t found[kMost];
    const int lane = threadIdx.x;
    const int64_t row = blockIdx.x;
    const int total = in.nseg * top;
    const uint64_t* list = lists + row * total;
    const int r = top > 0 ? (top + in.nseg - 1) / in.nseg : 1;
    // 0 past a segment's entries: such lists do not count
    const uint64_t mine = top > 0 && lane < in.nseg ? list[lane * top + r - 1] : 0;
    const Given t = given_token<kType>(in.logits + row * in.stride, in.vocab, row, out.targets);
    const ProbStats st = prob_stats(join_parts(part + row * in.nseg, in.nseg, in.c));
    if (lane == 0) write_prob(row, in.c, st, t, out);
    if (top == 0) return;
    const uint32_t want = (uint32_t)((top + r - 1) / r), key = (uint32_t)(mine >> 48);
    uint32_t bound = 0;
#pragma unroll
    for (int bit = 15; bit >= 0; --bit) {
        const uint32_t trial = bound | (1u << bit);
        if ((uint32_t)__popcll(__ballot(key >= trial)) >= want) bound = trial;
    }
    uint32_t n = 0;
    for (int at = 0; at < total; at += kWave) {
        const uint64_t e = at + lane < total ? list[at + lane] : 0;
        const bool is = e != 0 && (uint32_t)(e >> 48) >= bound;
        const uint64_t who = __ballot(is);
        const uint32_t k = n + __popcll(who & ((uint64_t(1) << lane) - 1));
        if (is && k < (uint32_t)kMost) found[k] = e;
        n += __popcll(who);
    }
    __syncthreads();
    if (n <= (uint32_t)kMost) {
        for (uint32_t q = lane; q < n; q += kWave) {
            const uint64_t x = found[q];
            uint32_t rank = 0;
#pragma unroll 4
            for (uint32_t j = 0; j < n; ++j) rank += found[j] > x ? 1u : 0u;
            if (rank < (uint32_t)top) write_top(out, row, top, (int)rank, x, in.c, st);
        }
    } else {
        // lane b walks the list of segment b (a row has at most 64)
        int at = 0;
        uint64_t head = lane < in.nseg ? list[lane * top] : 0;
        for (int k = 0; k < top; ++k) {
            const uint64_t best = wave_max_u64(head);
            if (head == best && lane < in.nseg) head = ++at < top ? list[lane * top + at] : 0;
            if (lane == 0) write_top(out, row, top, k, best, in.c, st);
        }
    }
}

// The gradient from stats (the backward call), or, with `part`, from the
// segments' parts of the same call, which the row's first block also writes
// out.
template <int kType, int kVecs, bool kEntropy>
__global__ __launch_bounds__(kBlock) void prob_grad_kernel(RowsIn<kType> in, ProbOut out,
                                                           const Part* part,
                                                           const ProbStats* stats,
                                                           ProbGrad<kType> G) {
    const Segment<kType> seg = in.segment(blockIdx.x);
    const Given t = given_token<kType>(seg.x, seg.vocab, seg.row, out.targets);
    const ProbStats st = part ? prob_stats(join_parts(part + seg.row * in.nseg, in.nseg, in.c))
                              : stats[seg.row];
    if (part && seg.begin == 0 && threadIdx.x == 0) write_prob(seg.row, in.c, st, t, out);
    prob_grad_segment<kType, kVecs, kEntropy>(seg, in.c, st, t, G);
}

// The list of a row as wave 0 holds it; the row's numbers of it for all.
template <int kType>
__device__ __forceinline__ void share_list(const Segment<kType>& seg, float c, const DistillIn& list,
                                           Listed& l, ListRow& shared) {
    l.id = -1;
    if (threadIdx.x < kWave) {
        const ListRow lr = list_row<kType>(seg.x, seg.vocab, seg.row, c, list, l);
        if (threadIdx.x == 0) shared = lr;
    }
}

template <int kType, int kVecs, bool kGrad>
__global__ __launch_bounds__(kBlock) void distill_kernel(RowsIn<kType> in, DistillIn list,
                                                         Part* part, float* loss,
                                                         DistillStats* stats,
                                                         DistillGrad<kType> G) {
    extern __shared__ uint32_t marks[];
    __shared__ Part red[kWavesPerBlock];
    __shared__ ListRow lr;
    const Segment<kType> seg = in.segment(blockIdx.x);
    const int words = seg.template chunks<kVecs>() * (kChunk<kType, kVecs> / 32);
    for (int i = threadIdx.x; i < words; i += kBlock) marks[i] = 0;
    __syncthreads();
    if (threadIdx.x < list.top) {
        const int64_t id = list.ids[seg.row * list.top + threadIdx.x];
        const int64_t at = id - seg.first_id();
        if (id >= seg.first_id() && id < seg.end_id()) atomicOr(&marks[at >> 5], 1u << (at & 31));
    }
    Listed l;
    l.id = -1;
    if (in.nseg == 1) share_list<kType>(seg, in.c, list, l, lr);
    __syncthreads();
    float mine;
    const Part p = segment_part<kType, kVecs, true, false>(seg, in.c, marks, nullptr, red, mine);
    if (in.nseg > 1) {
        if (threadIdx.x == 0) part[blockIdx.x] = p;
        return;
    }
    const DistillStats st = finish_row(p, lr, list.tail, in.c, in.c_low, l, seg.row, loss, stats, true);
    if (kGrad) distill_grad_segment<kType, kVecs>(seg, in.c, st, list.top, l, G);
}

// one wave a row
template <int kType>
__global__ __launch_bounds__(kWave) void distill_join_kernel(RowsIn<kType> in, DistillIn list,
                                                             const Part* part, float* loss,
                                                             DistillStats* stats) {
    const int64_t row = blockIdx.x;
    Listed l;
    const ListRow lr = list_row<kType>(in.logits + row * in.stride, in.vocab, row, in.c, list, l);
    finish_row(join_parts(part + row * in.nseg, in.nseg, in.c), lr, list.tail, in.c, in.c_low, l,
               row, loss, stats, true);
}

// As prob_grad_kernel.
template <int kType, int kVecs>
__global__ __launch_bounds__(kBlock) void distill_grad_kernel(RowsIn<kType> in, DistillIn list,
                                                              const Part* part, float* loss,
                                                              const DistillStats* stats,
                                                              DistillGrad<kType> G) {
    __shared__ ListRow lr;
    const Segment<kType> seg = in.segment(blockIdx.x);
    Listed l;
    DistillStats st;
    if (part) {
        share_list<kType>(seg, in.c, list, l, lr);
        __syncthreads();
        st = finish_row(join_parts(part + seg.row * in.nseg, in.nseg, in.c), lr, list.tail, in.c,
                        in.c_low, l, seg.row, loss, nullptr, seg.begin == 0);
    } else {
        st = stats[seg.row];
        list.tail = st.tail != 0.0f;
        share_list<kType>(seg, in.c, list, l, lr);
    }
    distill_grad_segment<kType, kVecs>(seg, in.c, st, list.top, l, G);
}

// ---- host ---------------------------------------------------------------------

// How a call cuts its rows.  A block streams a segment of a row.  A segment is the
// whole row (no join, one launch) from kBlocksWanted rows on, a block for each CU,
// and for rows of up to kWholeWords words: a launch takes 4 us of host time and the
// join 3 us of the GPU's.  Measured, the GPU's time of a graph's call, cut and
// whole, and a call's from the host: 32 rows of 16000 in BF16: 6.1 and 5.2 us, 17.3
// and 13.4; of 32000: 6.1 and 6.5, 17.2 and 13.4; of 65536: 6.6 and 11.3, 17.1 and
// 13.3.  At kWholeWords the host's time decides, at the cost of a replayed graph:
// a distillation's gradient of 32 rows of 32000 takes 9.8 us cut and 14.2 whole, from
// the host 18.3 and 14.4.  Top entries cost a cut row more: 32 rows of 50257, top 20:
// 16.8 and 14.2, 22.8 and 19.8; of 128256: 13.4 and 19.2.
//
// Longer rows, if few, are cut until 2 kBlocksWanted blocks run, with top entries
// kBlocksWanted (at most kMaxSegments a row, which one wave joins): 128256 entries
// with their gradient, one row: 7.0 us cut, 21.5 whole; 100 rows: 19.2 (21.0 with
// half the blocks) and 30.7; 200 rows: 31.8 (33.1) and 36.8; but the 64 best of 64 rows
// with twice the blocks 27.3 for 21.7, of 250 rows 38.1 for 31.9.  A segment is at most
// kMaxChunks chunks, whose maxima or marks lie in LDS.
//
// Chunks are the short ones where there are few of them, or where the last long
// one of a row that is one or two would be less than 3/4 full: 32 rows of 8000 in
// BF16: 4.4 us for 4.8, of 24000 6.4 for 6.2, but of 32000 7.4 for 6.5.
constexpr int64_t kBlocksWanted = 256, kWholeWords = 4096, kWholeWordsTop = 8192;
constexpr int kMaxChunks = 16;
struct Cut {
    int vecs;
    int64_t span;                                // 16-byte words of a segment
    int32_t nseg;
    int chunks;                                  // of a segment
};
static Cut cut_rows(int32_t type, int64_t rows, int64_t vocab, int32_t top) {
    const int64_t e = type == FLASHOPT_FP32 ? 4 : 8, words = (vocab + e - 1) / e;
    const int64_t step_long = kLong * kBlock, lng = (words + step_long - 1) / step_long;
    const bool whole = words <= (top > 0 ? kWholeWordsTop : kWholeWords);
    Cut k;
    k.vecs = kLong;
    if (whole ? lng <= 2 && (words - 1) % step_long < step_long * 3 / 4 : rows * lng < 256) k.vecs = kShort;
    const int64_t step = (int64_t)k.vecs * kBlock, chunks = (words + step - 1) / step;
    const int64_t blocks = top > 0 ? kBlocksWanted : 2 * kBlocksWanted;
    int64_t want = whole || rows >= kBlocksWanted ? 1 : (blocks + rows - 1) / (rows < 1 ? 1 : rows);
    if (want > kMaxSegments) want = kMaxSegments;
    k.chunks = (int)((chunks + want - 1) / want);
    if (k.chunks > kMaxChunks) k.chunks = kMaxChunks;
    k.span = k.chunks * step;
    k.nseg = (int32_t)((words + k.span - 1) / k.span);
    return k;
}

// a launch has less than 2^32 threads
static bool rows_fit(int32_t type, int64_t rows, int64_t vocab) {
    return rows <= FLASHOPT_ROWS_MAX && rows * cut_rows(type, rows, vocab, 0).nseg <= FLASHOPT_ROWS_MAX;
}

static int check_rows(const void* logits, int32_t type, int64_t rows, int64_t vocab, int64_t stride,
                      double temperature) {
    if (!valid_type(type)) return FLASHOPT_ERR_ARG;
    if (rows < 0 || vocab < 1 || vocab > FLASHOPT_VOCAB_MAX || stride < vocab ||
        stride > kMaxNumel || !rows_fit(type, rows, vocab))
        return FLASHOPT_ERR_SIZE;
    // 1/T and log2(e)/T are used as normal binary32 numbers
    if (!(temperature >= 0x1p-126) || !(temperature <= 0x1p126)) return FLASHOPT_ERR_ARG;
    if (rows == 0) return FLASHOPT_OK;
    if (!logits) return FLASHOPT_ERR_NULL;
    if (!aligned(logits, type_size(type))) return FLASHOPT_ERR_ALIGN;
    return FLASHOPT_OK;
}

// The gradient takes the logits' place exactly or shares nothing with them: rows
// are read again after others' gradients have been written.
static int check_grad(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                      int64_t stride, const void* grad, int64_t grad_stride) {
    if (!grad) return FLASHOPT_ERR_NULL;
    if (grad_stride < vocab || grad_stride > kMaxNumel) return FLASHOPT_ERR_SIZE;
    const int64_t size = (int64_t)type_size(type);
    if (!aligned(grad, size)) return FLASHOPT_ERR_ALIGN;
    const bool same = grad == logits && (grad_stride == stride || rows == 1);
    if (!same && overlap(rows, logits, stride * size, vocab * size, grad, grad_stride * size, vocab * size))
        return FLASHOPT_ERR_ARG;
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

// a row that one block holds needs no workspace
static size_t parts_bytes(const Cut& k, int64_t rows) {
    if (k.nseg == 1) return 0;
    const size_t b = (size_t)(rows * k.nseg) * sizeof(Part);
    return (b + 255) & ~size_t(255);
}
// and, for the gradient in the same call, stats behind the parts
static size_t both_bytes(const Cut& k, int64_t rows) {
    return k.nseg == 1 ? 0 : parts_bytes(k, rows) + (size_t)rows * sizeof(DistillStats);
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

template <int kType>
static ProbGrad<kType> prob_grad(const Rows& a, const Upstream& g) {
    return {g.logprob, g.entropy, (typename Elem<kType>::T*)g.grad, g.stride,
            (float)(1.0 / a.temperature)};
}
template <int kType>
static DistillGrad<kType> distill_grad(const Rows& a, const Upstream& g) {
    return {g.logprob, (typename Elem<kType>::T*)g.grad, g.stride, (float)(1.0 / a.temperature)};
}

// The gradient of cut rows: from stats, or from the parts of the same call.
static int launch_prob_grad(const Rows& a, const Cut& k, const ProbOut& out, const Part* part,
                            const float* stats, const Upstream& g, hipStream_t st) {
    return by_type(a.type, k.vecs, [&](auto t, auto v) {
        constexpr int kType = decltype(t)::value, kVecs = decltype(v)::value;
        const dim3 grid((unsigned)(a.rows * k.nseg));
        if (g.entropy)
            hipLaunchKernelGGL((prob_grad_kernel<kType, kVecs, true>), grid, dim3(kBlock), 0, st,
                               rows_in<kType>(a, k), out, part, (const ProbStats*)stats,
                               prob_grad<kType>(a, g));
        else
            hipLaunchKernelGGL((prob_grad_kernel<kType, kVecs, false>), grid, dim3(kBlock), 0, st,
                               rows_in<kType>(a, k), out, part, (const ProbStats*)stats,
                               prob_grad<kType>(a, g));
    });
}

static int launch_prob(const Rows& a, const ProbOut& out, int32_t top, void* workspace,
                       hipStream_t st) {
    const Cut k = cut_rows(a.type, a.rows, a.vocab, top);
    Part* part = (Part*)workspace;
    uint64_t* lists = (uint64_t*)((char*)workspace + parts_bytes(k, a.rows));
    return by_type(a.type, k.vecs, [&](auto t, auto v) {
        constexpr int kType = decltype(t)::value, kVecs = decltype(v)::value;
        const RowsIn<kType> in = rows_in<kType>(a, k);
        const dim3 grid((unsigned)(a.rows * k.nseg));
        const ProbGrad<kType> none = {};
        if (top > 0)
            hipLaunchKernelGGL((prob_kernel<kType, kVecs, true, 0>), grid, dim3(kBlock),
                               (size_t)k.chunks * kBlock * sizeof(float), st, in, out, top, part,
                               lists, none);
        else
            hipLaunchKernelGGL((prob_kernel<kType, kVecs, false, 0>), grid, dim3(kBlock), 0, st, in,
                               out, 0, part, lists, none);
        if (k.nseg > 1)
            hipLaunchKernelGGL((prob_join_kernel<kType>), dim3((unsigned)a.rows), dim3(kWave), 0, st,
                               in, out, top, part, lists);
    });
}

static int launch_prob_both(const Rows& a, const ProbOut& out, void* workspace, const Upstream& g,
                            hipStream_t st) {
    if (launch_rows_prob(a, out, g, st)) return launch_status();
    const Cut k = cut_rows(a.type, a.rows, a.vocab, 0);
    Part* part = (Part*)workspace;
    const int f = by_type(a.type, k.vecs, [&](auto t, auto v) {
        constexpr int kType = decltype(t)::value, kVecs = decltype(v)::value;
        const RowsIn<kType> in = rows_in<kType>(a, k);
        const dim3 grid((unsigned)(a.rows * k.nseg));
        const ProbGrad<kType> G = prob_grad<kType>(a, g);
        if (k.nseg > 1)
            hipLaunchKernelGGL((prob_kernel<kType, kVecs, false, 0>), grid, dim3(kBlock), 0, st, in,
                               out, 0, part, nullptr, G);
        else if (g.entropy)
            hipLaunchKernelGGL((prob_kernel<kType, kVecs, false, 2>), grid, dim3(kBlock), 0, st, in,
                               out, 0, part, nullptr, G);
        else
            hipLaunchKernelGGL((prob_kernel<kType, kVecs, false, 1>), grid, dim3(kBlock), 0, st, in,
                               out, 0, part, nullptr, G);
    });
    if (f || k.nseg == 1) return f;
    if (g.grad != a.logits) return launch_prob_grad(a, k, out, part, nullptr, g, st);
    // A gradient in the logits' place: a segment's block would replace the given
    // token's logit before the row's first block has read it.  So the row is
    // finished by a launch of its own.
    ProbOut first = out, none = {out.targets, nullptr, nullptr, nullptr, nullptr, nullptr};
    first.stats = (ProbStats*)((char*)workspace + parts_bytes(k, a.rows));
    by_type(a.type, k.vecs, [&](auto t, auto) {
        constexpr int kType = decltype(t)::value;
        hipLaunchKernelGGL((prob_join_kernel<kType>), dim3((unsigned)a.rows), dim3(kWave), 0, st,
                           rows_in<kType>(a, k), first, 0, part, nullptr);
    });
    return launch_prob_grad(a, k, none, nullptr, (const float*)first.stats, g, st);
}

static int launch_distill_grad(const Rows& a, const Cut& k, const DistillIn& list,
                               const Part* part, float* loss, const float* stats,
                               const Upstream& g, hipStream_t st) {
    return by_type(a.type, k.vecs, [&](auto t, auto v) {
        constexpr int kType = decltype(t)::value, kVecs = decltype(v)::value;
        hipLaunchKernelGGL((distill_grad_kernel<kType, kVecs>), dim3((unsigned)(a.rows * k.nseg)),
                           dim3(kBlock), 0, st, rows_in<kType>(a, k), list, part, loss,
                           (const DistillStats*)stats, distill_grad<kType>(a, g));
    });
}

// grad null: the forward pass alone
static int launch_distill(const Rows& a, const DistillIn& list, void* workspace, float* loss,
                          float* stats, const Upstream& g, hipStream_t st) {
    const Cut k = cut_rows(a.type, a.rows, a.vocab, 0);
    Part* part = (Part*)workspace;
    const int f = by_type(a.type, k.vecs, [&](auto t, auto v) {
        constexpr int kType = decltype(t)::value, kVecs = decltype(v)::value;
        const RowsIn<kType> in = rows_in<kType>(a, k);
        const dim3 grid((unsigned)(a.rows * k.nseg));
        const DistillGrad<kType> G = distill_grad<kType>(a, g);
        const size_t lds = (size_t)k.chunks * kChunk<kType, kVecs> / 8;
        if (g.grad && k.nseg == 1)
            hipLaunchKernelGGL((distill_kernel<kType, kVecs, true>), grid, dim3(kBlock), lds, st, in,
                               list, part, loss, (DistillStats*)stats, G);
        else
            hipLaunchKernelGGL((distill_kernel<kType, kVecs, false>), grid, dim3(kBlock), lds, st, in,
                               list, part, loss, (DistillStats*)stats, G);
        // (a gradient in the logits' place: as in launch_prob_both)
        if (k.nseg > 1 && (!g.grad || g.grad == a.logits)) {
            if (g.grad) stats = (float*)((char*)workspace + parts_bytes(k, a.rows));
            hipLaunchKernelGGL((distill_join_kernel<kType>), dim3((unsigned)a.rows), dim3(kWave), 0,
                               st, in, list, part, loss, (DistillStats*)stats);
        }
    });
    if (f || k.nseg == 1 || !g.grad) return f;
    if (g.grad == a.logits) return launch_distill_grad(a, k, list, nullptr, nullptr, stats, g, st);
    return launch_distill_grad(a, k, list, part, loss, nullptr, g, st);
}

}  // namespace flashopt

using namespace flashopt;

extern "C" {

size_t flashopt_logprob_workspace_bytes(int32_t type, int64_t rows, int64_t vocab, int32_t top) {
    if (!valid_type(type) || rows < 0 || vocab < 1 || vocab > FLASHOPT_VOCAB_MAX || top < 0 ||
        top > FLASHOPT_TOP_MAX || !rows_fit(type, rows, vocab))
        return 0;
    // the forward call's and, so that one workspace serves both, the gradient's
    const Cut k = cut_rows(type, rows, vocab, top);
    const size_t lists = k.nseg == 1 ? 0 : (size_t)(rows * k.nseg) * (size_t)top * sizeof(uint64_t);
    const size_t forward = parts_bytes(k, rows) + lists, both = both_bytes(cut_rows(type, rows, vocab, 0), rows);
    return forward > both ? forward : both;
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
                       workspace, (hipStream_t)stream);
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
    const int g = check_grad(logits, type, rows, vocab, stride, grad, grad_stride);
    if (g) return g;
    return launch_prob_grad({logits, type, rows, vocab, stride, temperature},
                            cut_rows(type, rows, vocab, 0),
                            {targets, nullptr, nullptr, nullptr, nullptr, nullptr}, nullptr, stats,
                            {grad_logprob, grad_entropy, grad, grad_stride}, (hipStream_t)stream);
}

int flashopt_logprob_grad(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                          int64_t stride, double temperature, const int64_t* targets,
                          const float* grad_logprob, const float* grad_entropy, void* workspace,
                          size_t workspace_bytes, float* logprob, float* entropy, void* grad,
                          int64_t grad_stride, void* stream) {
    const int e = check_rows(logits, type, rows, vocab, stride, temperature);
    if (e) return e;
    if (rows == 0) return FLASHOPT_OK;
    if ((logprob || grad_logprob) && !targets) return FLASHOPT_ERR_NULL;
    if (!aligned(targets, 8) || !aligned(logprob, 4) || !aligned(entropy, 4) ||
        !aligned(grad_logprob, 4) || !aligned(grad_entropy, 4))
        return FLASHOPT_ERR_ALIGN;
    const int g = check_grad(logits, type, rows, vocab, stride, grad, grad_stride);
    if (g) return g;
    const int w = check_workspace(workspace, workspace_bytes,
                                  flashopt_logprob_workspace_bytes(type, rows, vocab, 0));
    if (w) return w;
    return launch_prob_both({logits, type, rows, vocab, stride, temperature},
                            {targets, logprob, entropy, nullptr, nullptr, nullptr}, workspace,
                            {grad_logprob, grad_entropy, grad, grad_stride}, (hipStream_t)stream);
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
                          {top_id, top_logprob, top, tail}, workspace, loss, stats, {},
                          (hipStream_t)stream);
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
    const int g = check_grad(logits, type, rows, vocab, stride, grad, grad_stride);
    if (g) return g;
    return launch_distill_grad({logits, type, rows, vocab, stride, temperature},
                               cut_rows(type, rows, vocab, 0), {top_id, top_logprob, top, 0}, nullptr,
                               nullptr, stats, {grad_loss, nullptr, grad, grad_stride},
                               (hipStream_t)stream);
}

int flashopt_distill_grad(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                          int64_t stride, double temperature, const int64_t* top_id,
                          const float* top_logprob, int32_t top, int32_t tail,
                          const float* grad_loss, void* workspace, size_t workspace_bytes,
                          float* loss, void* grad, int64_t grad_stride,
                          void* stream) {
    const int e = check_rows(logits, type, rows, vocab, stride, temperature);
    if (e) return e;
    if (top < 1 || top > FLASHOPT_TOP_MAX || top > vocab || tail < 0 || tail > 1)
        return FLASHOPT_ERR_ARG;
    if (rows == 0) return FLASHOPT_OK;
    const int l = check_list(top_id, top_logprob, top, vocab);
    if (l) return l;
    if (!grad_loss) return FLASHOPT_ERR_NULL;
    if (!aligned(loss, 4) || !aligned(grad_loss, 4)) return FLASHOPT_ERR_ALIGN;
    const int g = check_grad(logits, type, rows, vocab, stride, grad, grad_stride);
    if (g) return g;
    const int w = check_workspace(workspace, workspace_bytes,
                                  flashopt_distill_workspace_bytes(type, rows, vocab));
    if (w) return w;
    return launch_distill({logits, type, rows, vocab, stride, temperature},
                          {top_id, top_logprob, top, tail}, workspace, loss, nullptr,
                          {grad_loss, nullptr, grad, grad_stride}, (hipStream_t)stream);
}

}  // extern "C"
