// Rows of logits: the device code that logits.hip (rows in segments) and
// logits_row.hip (whole rows in registers) share.
#pragma once

#include "rows.hpp"

namespace flashopt {

// A part of a row: maximum of x, S, U.
struct Part {
    float m, s, u, pad;
};

// The largest entry of N words.  16-bit types are compared as pairs of integers:
// those order like the numbers where one is not negative, and against them where
// all are.  (NaN and infinities of either sign may be the result where the words
// hold a NaN.)  2 slots a pair of entries less than unpacked.
template <int kType, int N>
__device__ __forceinline__ float largest(const u32x4* r) {
    if constexpr (kType == FLASHOPT_FP32) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) m = fmaxf(m, as_f32(r[i][e]));
        return m;
    } else {
        typedef int16_t I2 __attribute__((ext_vector_type(2)));
        typedef uint16_t U2 __attribute__((ext_vector_type(2)));
        const uint32_t first = r[0][0];          // (__builtin_bit_cast takes no element of a vector)
        I2 a = __builtin_bit_cast(I2, first);
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t w = r[i][q];
                a = __builtin_elementwise_max(a, __builtin_bit_cast(I2, w));
            }
        int top = max((int)a[0], (int)a[1]);
        if (top < 0) {
            U2 b = __builtin_bit_cast(U2, first);
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t w = r[i][q];
                    b = __builtin_elementwise_min(b, __builtin_bit_cast(U2, w));
                }
            top = min((int)b[0], (int)b[1]);
        }
        return Elem<kType>::up((uint16_t)top);
    }
}

// A sum of up to 16 numbers by pairs, pairs of pairs and so on; i counts them, as
// an unrolled loop's constant.
struct PairSum {
    float level[5];
    __device__ __forceinline__ void add(int i, float x) {
        int k = 0;
#pragma unroll
        for (; k < 4 && (i >> k & 1); ++k) x = level[k] + x;
        level[k] = x;
    }
    __device__ __forceinline__ float total(int n) const {
        float x = 0.0f;
        bool any = false;
#pragma unroll
        for (int k = 0; k < 5; ++k)
            if (n >> k & 1) {
                x = any ? level[k] + x : level[k];
                any = true;
            }
        return x;
    }
};

// ---- parts --------------------------------------------------------------------------

// The parts of a wave's threads as one (every lane gets it).
template <bool kU>
__device__ __forceinline__ Part wave_part(float m, float s, float u, float c) {
    const float wm = wave_max(m);
    const float D = fmaxf((m - wm) * c, -200.0f), f = exp2_hw(D);
    return Part{wm, wave_sum(s * f), kU ? wave_sum(f * (u + D * s)) : 0.0f, 0.0f};
}

// n parts as one (one wave; every lane gets it).
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

// Two parts as one, without their u.
__device__ __forceinline__ Part add_parts(const Part& a, const Part& b, float c) {
    const bool no_a = a.m == -INFINITY && a.s == 0.0f, no_b = b.m == -INFINITY && b.s == 0.0f;
    const float m = fmaxf(a.m, b.m);
    const float fa = no_a ? 0.0f : a.s * exp2_hw(fmaxf((a.m - m) * c, -200.0f));
    const float fb = no_b ? 0.0f : b.s * exp2_hw(fmaxf((b.m - m) * c, -200.0f));
    return Part{m, fa + fb, 0.0f, 0.0f};
}

// ---- a row's log probabilities ----------------------------------------------------------

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

// A row's given token and its logit (0 for none).
struct Given {
    int64_t id;                                  // -1: none
    float x;
};
template <int kType>
__device__ __forceinline__ Given given_token(const typename Elem<kType>::T* x, int64_t vocab,
                                             int64_t row, const int64_t* targets) {
    Given g = {targets ? targets[row] : -1, 0.0f};
    if (g.id < 0 || g.id >= vocab) g.id = -1;
    else g.x = Elem<kType>::up(x[g.id]);
    return g;
}

// The given token's gradient gl (1 - p) - gh p (log p + H), with 1 - p from its
// logarithm: p itself is near 1 where it matters.
template <bool kEntropy>
__device__ __forceinline__ float given_grad(float x, const ProbStats& st, float c, float gl, float gh) {
    const float d = (x - st.m) * c - st.l2s, y = d * kLn2, p = exp2_hw(d);
    float rest = 1.0f - p;
    if (y > -0.25f) {                            // -(e^y - 1): the next term is below 2^-29 of it
        float t = __builtin_fmaf(y, 1.0f / 7, 1.0f);
        t = __builtin_fmaf(y * (1.0f / 6), t, 1.0f);
        t = __builtin_fmaf(y * (1.0f / 5), t, 1.0f);
        t = __builtin_fmaf(y * (1.0f / 4), t, 1.0f);
        t = __builtin_fmaf(y * (1.0f / 3), t, 1.0f);
        t = __builtin_fmaf(y * (1.0f / 2), t, 1.0f);
        rest = -y * t;
    }
    float v = gl * rest;
    if (kEntropy) v -= gh * (p * (fmaxf(y, -140.0f) + st.entropy));
    return v;
}

// one lane
__device__ __forceinline__ void write_prob(int64_t row, float c, const ProbStats& st,
                                           const Given& g, const ProbOut& o) {
    if (o.entropy) o.entropy[row] = st.entropy;
    if (o.stats) o.stats[row] = st;
    if (o.logprob) o.logprob[row] = g.id >= 0 ? ((g.x - st.m) * c - st.l2s) * kLn2 : 0.0f;
}

// ---- a row of distillation --------------------------------------------------------------

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
// a * b as a rounded product and what that leaves, with b = b + b_low
__device__ __forceinline__ void product_parts(float a, float b, float b_low, float& hi, float& lo) {
    hi = a * b;
    lo = __builtin_fmaf(a, b, -hi) + a * b_low;
    if (!(__builtin_fabsf(hi) < 3e38f)) lo = 0.0f;               // no inf - inf
}
constexpr float kLog2eLow = 0x1.4ae0cp-26f;      // 1 / log 2 - kLog2e

// One lane's alternative, as wave 0 of a block (or a wave of a join) holds it.
struct Listed {
    int id;                                      // -1: none
    float x;                                     // the student's logit
    float hi, lo;                                // log2 of q before its norm, from the list's base
    float q;
};
// The list's numbers of a row, equal in all lanes: the part of its entries (a
// repeated id once), Q, the teacher's norm (0 with a tail) as log2, from the base.
// Without a tail the base is the whole part of the list's largest number, so that
// q means the same wherever a list lies; with one it is 0.
struct ListRow {
    Part part;
    float Q, norm_whole, norm_frac, any;
};

// q = 2^(hi + lo - norm): whole parts go into the exponent, so that a small q
// is good to its last bits too
__device__ __forceinline__ float list_q(const Listed& l, float nwhole, float nfrac) {
    if (l.hi <= -300.0f) return 0.0f;
    const float n = __builtin_rintf(l.hi);
    return __builtin_amdgcn_ldexpf(exp2_hw((l.hi - n) + (l.lo - nfrac)), (int)(n - nwhole));
}

template <int kType>
__device__ __forceinline__ ListRow list_row(const typename Elem<kType>::T* x, int64_t vocab,
                                            int64_t row, float c, const DistillIn& in, Listed& l) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t id = lane < in.top ? in.ids[row * in.top + lane] : -1;
    float t = lane < in.top ? in.tlp[row * in.top + lane] : 0.0f;
    const bool ok = id >= 0 && id < vocab;
    l.id = ok ? (int)id : -1;
    l.x = ok ? Elem<kType>::up(x[l.id]) : -INFINITY;
    if (!ok) t = -INFINITY;
    product_parts(t, kLog2e, kLog2eLow, l.hi, l.lo);
    bool first = ok;
    for (int k = 0; k < in.top - 1; ++k) {
        const int other = __builtin_amdgcn_readlane(l.id, k);
        if (k < lane && other == l.id) first = false;
    }
    ListRow r;
    r.part = wave_part<false>(first ? l.x : -INFINITY, first && !(l.x == -INFINITY) ? 1.0f : 0.0f, 0.0f, c);
    if (__ballot(ok && !(l.x < INFINITY))) r.part.s = NAN;       // NaN or +inf
    r.norm_whole = r.norm_frac = 0.0f;
    if (!in.tail) {
        const float tm = wave_max(t);
        const float ts = wave_sum(ok ? exp2_hw((t - tm) * kLog2e) : 0.0f);
        float hi, lo, f;
        product_parts(tm, kLog2e, kLog2eLow, hi, lo);
        log2_parts(ts, r.norm_whole, f);
        const float base = tm == -INFINITY ? 0.0f : __builtin_rintf(hi);     // (nothing but -inf: q = 0)
        r.norm_frac = (hi - base) + (lo + f);
        l.hi -= base;
    }
    l.q = ok ? list_q(l, r.norm_whole, r.norm_frac) : 0.0f;
    r.Q = wave_sum(l.q);
    r.any = __ballot(ok) ? 1.0f : 0.0f;
    return r;
}

// stats of a row.  The gradient is
//   outside the list: e_j coef, e_j = 2^((x_j - rest_m) c - rest_l2) the
//                     entry's share of the rest, coef = (Q + r) P - r;
//   in the list:      (Q + r) p_j - sum of its q, p_j from m and l2s;
// q from the list again, with its tail or without (1 or 0), all times g / T.  A
// row without a gradient has on = 0.
struct DistillStats {
    float rest_m, rest_l2, coef, qr, m, l2s, tail, on;
};

// The row's numbers from the part of its unlisted entries; `loss`, with each
// lane's alternative, is the row's in every lane of a wave.  The divergence is
// a difference of logarithms near 10 that may itself be near 0: their whole
// parts are subtracted exactly.
__device__ __forceinline__ DistillStats distill_stats(const Part& rest, const ListRow& lr, int tail,
                                                      float c, float c_low, bool want_loss,
                                                      const Listed& l, float& loss) {
    const Part all = add_parts(rest, lr.part, c);
    const bool no_rest = rest.m == -INFINITY && rest.s == 0.0f;
    const bool empty = all.m == -INFINITY && all.s == 0.0f;      // no distribution
    const float m = empty ? 0.0f : all.m, rest_m = no_rest ? 0.0f : rest.m;
    float sw = 0.0f, sf = 0.0f, rw = 0.0f, rf = 0.0f;
    if (!empty) log2_parts(all.s, sw, sf);
    if (!no_rest) log2_parts(rest.s, rw, rf);
    const float r = tail && !no_rest ? fmaxf(0.0f, 1.0f - lr.Q) : 0.0f;
    float dh, dl;
    product_parts(rest_m - m, c, c_low, dh, dl);
    const float P = no_rest ? 0.0f : exp2_hw((dh + (rw - sw)) + (dl + (rf - sf)));
    const bool on = lr.any != 0.0f && !empty;
    if (want_loss) {
        float term = 0.0f;
        if (l.q > 0.0f) {                        // log2 q - log2 p
            float ph, pl;
            product_parts(l.x - m, c, c_low, ph, pl);
            term = l.q * (((l.hi - ph) + (sw - lr.norm_whole)) + ((l.lo - pl) + (sf - lr.norm_frac)));
        } else if (l.q != 0.0f) {
            term = l.q;                          // NaN
        }
        float sum = wave_sum(term);
        if (r > 0.0f) {
            float w, f;
            log2_parts(r, w, f);
            sum += r * (((w - rw) + sw - dh) + ((f - rf) + (sf - dl)));
        }
        loss = on ? sum * kLn2 : 0.0f;
    }
    return DistillStats{rest_m, rw + rf, on ? (lr.Q + r) * P - r : 0.0f, lr.Q + r, m, sw + sf,
                        (float)tail, on ? 1.0f : 0.0f};
}

// One lane's alternative's gradient (wave 0); w = g / T, 0 where on = 0.
__device__ __forceinline__ float listed_grad(const Listed& l, const DistillStats& st, int top,
                                             float c, float w) {
    float sum = 0.0f;
    for (int k = 0; k < top; ++k) {
        const int other = __builtin_amdgcn_readlane(l.id, k);
        const float q = as_f32((uint32_t)__builtin_amdgcn_readlane((int)as_u32(l.q), k));
        if (other == l.id) sum += q;
    }
    const float p = exp2_hw((l.x - st.m) * c - st.l2s);
    return st.on != 0.0f ? w * (st.qr * p - sum) : 0.0f;
}

// ---- finishing a row ------------------------------------------------------------------

// Stats from the rest's part for every thread; wave 0 forms the loss.
__device__ __forceinline__ DistillStats finish_row(const Part& rest, const ListRow& lr, int tail,
                                                   float c, float c_low, const Listed& l,
                                                   int64_t row, float* loss, DistillStats* stats,
                                                   bool write) {
    float v = 0.0f;
    const bool wave0 = threadIdx.x < kWave && write;
    const DistillStats st = distill_stats(rest, lr, tail, c, c_low, wave0, l, v);
    if (wave0 && threadIdx.x == 0) {
        if (loss) loss[row] = v;
        if (stats) stats[row] = st;
    }
    return st;
}

// ---- calls ------------------------------------------------------------------------------

struct Rows {                                    // a call's logits
    const void* logits;
    int32_t type;
    int64_t rows, vocab, stride;
    double temperature;
};
struct Upstream {                                // and where the gradient goes
    const float *logprob, *entropy;              // of distillation: loss, null
    void* grad;
    int64_t stride;
};

// logits_row.hip: log probability and gradient of rows that fit a block's
// registers; false if these rows are to be cut into segments instead.
bool launch_rows_prob(const Rows& a, const ProbOut& out, const Upstream& g, hipStream_t st);

}  // namespace flashopt
