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

constexpr int kVecs = 8;                         // 16-byte words of a chunk per thread
constexpr int kChunkVecs = kVecs * kBlock;
template <int kType> constexpr int kChunk = kChunkVecs * Elem<kType>::kE;

static int chunk_of(int32_t type) {
    return type == FLASHOPT_FP32 ? kChunk<FLASHOPT_FP32> : kChunk<FLASHOPT_BF16>;
}
static int64_t chunks_of(int32_t type, int64_t vocab) {
    const int64_t c = chunk_of(type);
    return (vocab + c - 1) / c;
}

// One chunk's numbers: maximum of x, S, U.
struct Part {
    float m, s, u, pad;
};

// A row's order of entries as unsigned numbers: larger logit first, equal
// ones by lowest id; a NaN ranks above all.  key: the value's order as 32
// bits (16-bit types use the upper half).
template <int kType>
__device__ __forceinline__ uint32_t order_key(const u32x4& v, int e) {
    uint32_t b;
    if (kType == FLASHOPT_FP32) b = v[e & 3];
    else b = ((e & 1) ? v[e >> 1] & 0xFFFF0000u : v[e >> 1] << 16);
    constexpr uint32_t kInf = kType == FLASHOPT_FP16 ? 0x7C000000u : 0x7F800000u;
    const uint32_t mag = b & 0x7FFFFFFFu;
    if (mag > kInf) return kType == FLASHOPT_FP32 ? 0xFFFFFFFFu : 0xFFFF0000u;
    if (mag == 0) b = 0;                         // -0 equals +0
    return (b & 0x80000000u) ? ~b & (kType == FLASHOPT_FP32 ? 0xFFFFFFFFu : 0xFFFF0000u)
                             : b | 0x80000000u;
}
template <int kType>
__device__ __forceinline__ float key_value(uint32_t k) {
    uint32_t b = (k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k;
    if (kType == FLASHOPT_FP32) return as_f32(b);
    b >>= 16;
    return Elem<kType>::up((typename Elem<kType>::T)b);
}

__device__ __forceinline__ uint64_t entry(uint32_t key, uint32_t id) {
    return ((uint64_t)key << 32) | (0xFFFFFFFFu - id);   // never 0 for an id that exists
}
__device__ __forceinline__ uint32_t entry_id(uint64_t e) { return 0xFFFFFFFFu - (uint32_t)e; }
__device__ __forceinline__ uint32_t entry_key(uint64_t e) { return (uint32_t)(e >> 32); }

template <int kType>
__device__ __forceinline__ void load_chunk(const typename Elem<kType>::T* row, int64_t vocab,
                                           int64_t v0, u32x4* r) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
        r[i] = load_vec<kType>(row, v0 + i * kBlock, vocab, Elem<kType>::kMinusInf);
}

// The `top` best entries of a chunk, best first, into list[0, top); places
// past the chunk's entries get 0.  The smallest entry wanted is found by
// halving: an entry is its key and its place in the chunk as one number, so
// all differ, and the bits of the top-th largest are set from the highest
// down by counting the entries at or above each trial.
template <int kType>
__device__ void chunk_top(const u32x4* r, int64_t v0, int64_t vocab, int top, uint64_t* list) {
    constexpr int E = Elem<kType>::kE;
    __shared__ uint32_t count[2][kWavesPerBlock];
    __shared__ uint64_t found[FLASHOPT_TOP_MAX];
    __shared__ uint32_t nfound;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t left = vocab - (v0 - threadIdx.x) * E;         // the row's entries from here
    const uint32_t here = left < kChunk<kType> ? (uint32_t)left : (uint32_t)kChunk<kType>;
    const uint32_t need = min((uint32_t)top, here);
    if (threadIdx.x == 0) nfound = 0;
    uint64_t bound = 0;
    int turn = 0;
    for (int bit = 63; bit >= 0; --bit) {
        if (bit < 32 && bit >= 20) {             // ids are below 2^20: these bits are set
            bound |= uint64_t(1) << bit;
            continue;
        }
        if (kType != FLASHOPT_FP32 && bit < 48 && bit >= 32) continue;   // and these clear
        const uint64_t trial = bound | (uint64_t(1) << bit);
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int64_t id = (v0 + i * kBlock) * E + e;
                const bool in = id < vocab && entry(order_key<kType>(r[i], e), (uint32_t)id) >= trial;
                n += __popcll(__ballot(in));
            }
        if (lane == 0) count[turn][wave] = n;
        __syncthreads();
        uint32_t all = 0;
#pragma unroll
        for (int w = 0; w < kWavesPerBlock; ++w) all += count[turn][w];
        turn ^= 1;
        if (all >= need) bound = trial;
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t id = (v0 + i * kBlock) * E + e;
            const uint64_t x = entry(order_key<kType>(r[i], e), (uint32_t)id);
            if (id < vocab && x >= bound) {
                const uint32_t at = atomicAdd(&nfound, 1u);
                if (at < FLASHOPT_TOP_MAX) found[at] = x;
            }
        }
    __syncthreads();
    if (threadIdx.x < top) {
        if (threadIdx.x >= need) {
            list[threadIdx.x] = 0;
        } else {
            const uint64_t x = found[threadIdx.x];
            uint32_t rank = 0;
            for (uint32_t k = 0; k < need; ++k) rank += found[k] > x ? 1u : 0u;
            list[rank] = x;
        }
    }
}

// ---- forward: a chunk ---------------------------------------------------------

// One block per chunk of a row.  kListed: the row's `top` ids are left out of
// the sums (distillation: the sums are those of the rest), marked in a
// bitmap of the chunk, one byte (16-bit types) or nibble per 16-byte word.
template <int kType, bool kListed, bool kTop>
__global__ __launch_bounds__(kBlock) void chunk_kernel(
    const typename Elem<kType>::T* logits, int64_t vocab, int64_t stride, int32_t nchunk, float c,
    const int64_t* ids, int top, Part* part, uint64_t* lists) {
    constexpr int E = Elem<kType>::kE;
    const int64_t row = blockIdx.x / nchunk;
    const int64_t chunk = blockIdx.x % nchunk;
    const typename Elem<kType>::T* x = logits + row * stride;
    const int64_t v0 = chunk * kChunkVecs + threadIdx.x;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    __shared__ uint32_t marks[kListed ? kChunk<kType> / 32 : 1];
    __shared__ float red[kWavesPerBlock][3];
    u32x4 r[kVecs];
    load_chunk<kType>(x, vocab, v0, r);
    if (kListed) {
        for (int i = threadIdx.x; i < kChunk<kType> / 32; i += kBlock) marks[i] = 0;
        __syncthreads();
        if (threadIdx.x < top) {
            const int64_t id = ids[row * top + threadIdx.x] - chunk * kChunk<kType>;
            if (id >= 0 && id < kChunk<kType>) atomicOr(&marks[id >> 5], 1u << (id & 31));
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int at = (i * kBlock + (int)threadIdx.x) * E;
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
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) m = fmaxf(m, Elem<kType>::get(r[i], e));
    m = wave_max(m);
    const float shift = m == -INFINITY ? 0.0f : m;       // nothing here: every e_j is 0
    float s = 0.0f, u = 0.0f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float d = (Elem<kType>::get(r[i], e) - shift) * c;
            const float p = exp2_hw(d);
            s += p;
            // p is 0 below -150: the bound keeps 0 * -inf out of the sum
            if (!kListed) u = __builtin_fmaf(p, fmaxf(d, -200.0f), u);
        }
    s = wave_sum(s);
    if (!kListed) u = wave_sum(u);
    if (lane == 0) { red[wave][0] = m; red[wave][1] = s; red[wave][2] = u; }
    __syncthreads();
    if (threadIdx.x == 0) {
        float M = red[0][0], S = 0.0f, U = 0.0f;
        for (int w = 1; w < kWavesPerBlock; ++w) M = fmaxf(M, red[w][0]);
        for (int w = 0; w < kWavesPerBlock; ++w) {
            if (red[w][0] == -INFINITY && red[w][1] == 0.0f) continue;   // an empty part
            const float D = fmaxf((red[w][0] - M) * c, -200.0f), f = exp2_hw(D);
            S += red[w][1] * f;
            U += f * (red[w][2] + D * red[w][1]);
        }
        part[blockIdx.x] = Part{M, S, U, 0.0f};
    }
    if (kTop) chunk_top<kType>(r, v0, vocab, top, lists + (int64_t)blockIdx.x * top);
}

// ---- forward: a row -----------------------------------------------------------

// The row's numbers from its chunks' (one wave; every lane gets them).
__device__ __forceinline__ Part join_parts(const Part* part, int32_t nchunk, float c) {
    const int lane = threadIdx.x & (kWave - 1);
    float m = -INFINITY;
    for (int k = lane; k < nchunk; k += kWave) m = fmaxf(m, part[k].m);
    m = wave_max(m);
    float s = 0.0f, u = 0.0f;
    for (int k = lane; k < nchunk; k += kWave) {
        const Part p = part[k];
        if (p.m == -INFINITY && p.s == 0.0f) continue;
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

template <int kType>
__global__ __launch_bounds__(kBlock) void logprob_join_kernel(
    const typename Elem<kType>::T* logits, int64_t rows, int64_t vocab, int64_t stride,
    int32_t nchunk, float c, const int64_t* targets, int top, const Part* part,
    const uint64_t* lists, float* logprob, float* entropy, ProbStats* stats, float* top_logprob,
    int64_t* top_id) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t row = (int64_t)blockIdx.x * kWavesPerBlock + threadIdx.x / kWave;
    if (row >= rows) return;
    Part p = join_parts(part + row * nchunk, nchunk, c);
    const bool empty = p.m == -INFINITY && p.s == 0.0f;
    const float m = empty ? 0.0f : p.m;
    const float l2s = empty ? 0.0f : log2_hw(p.s);
    const float h = empty ? 0.0f : (l2s - p.u / p.s) * kLn2;
    if (lane == 0) {
        if (entropy) entropy[row] = h;
        if (stats) stats[row] = ProbStats{m, l2s, h, empty ? 0.0f : 1.0f};
        if (logprob) {
            const int64_t t = targets[row];
            float lp = 0.0f;
            if (t >= 0 && t < vocab)
                lp = ((Elem<kType>::up(logits[row * stride + t]) - m) * c - l2s) * kLn2;
            logprob[row] = lp;
        }
    }
    if (top > 0) {
        // lane b walks the list of chunk b, best first (vocab is at most 64 chunks)
        const uint64_t* mine = lists + (row * nchunk + lane) * top;
        int at = 0;
        uint64_t head = lane < nchunk ? mine[0] : 0;
        for (int k = 0; k < top; ++k) {
            const uint64_t best = wave_max_u64(head);
            if (head == best && lane < nchunk) head = ++at < top ? mine[at] : 0;
            if (lane == 0) {
                top_id[row * top + k] = entry_id(best);
                top_logprob[row * top + k] =
                    ((key_value<kType>(entry_key(best)) - m) * c - l2s) * kLn2;
            }
        }
    }
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

template <int kType>
__global__ __launch_bounds__(kBlock) void distill_join_kernel(
    const typename Elem<kType>::T* logits, int64_t rows, int64_t vocab, int64_t stride,
    int32_t nchunk, float c, const int64_t* ids, const float* tlp, int top, int tail,
    const Part* part, float* loss, DistillStats* stats) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t row = (int64_t)blockIdx.x * kWavesPerBlock + threadIdx.x / kWave;
    if (row >= rows) return;
    const Part rest = join_parts(part + row * nchunk, nchunk, c);
    // lane k holds alternative k; a repeated id is summed into P once
    const int64_t id = lane < top ? ids[row * top + lane] : -1;
    const bool in = id >= 0 && id < vocab;
    const float x = in ? Elem<kType>::up(logits[row * stride + id]) : -INFINITY;
    const float t = in ? tlp[row * top + lane] : -INFINITY;
    bool first = in;
    for (int k = 0; k < top - 1; ++k) {
        const int64_t other = __shfl((long long)id, k);
        if (k < lane && other == id) first = false;
    }
    const float m0 = fmaxf(rest.m, wave_max(x));
    const bool any_in = __ballot(in) != 0;
    const bool no_rest = rest.m == -INFINITY && rest.s == 0.0f;
    // the student's row has no distribution
    const bool empty = m0 == -INFINITY && no_rest && __ballot(in && x != x) == 0;
    const float m = empty ? 0.0f : m0;
    const float rest_f = no_rest ? 0.0f : exp2_hw(fmaxf((rest.m - m) * c, -200.0f));
    const float s = wave_sum(first ? exp2_hw((x - m) * c) : 0.0f) + (no_rest ? 0.0f : rest.s * rest_f);
    const float l2s = empty ? 0.0f : log2_hw(s);
    // the teacher's side
    float norm = 0.0f;
    if (!tail) {
        const float tm = wave_max(t);
        const float ts = wave_sum(in ? exp2_hw((t - tm) * kLog2e) : 0.0f);
        norm = tm * kLog2e + log2_hw(ts);
    }
    const float l2q = in ? t * kLog2e - norm : -INFINITY;
    const float q = in ? exp2_hw(l2q) : 0.0f;
    const float Q = wave_sum(q);
    float r = tail ? fmaxf(0.0f, 1.0f - Q) : 0.0f;
    if (no_rest) r = 0.0f;
    const float l2p = (x - m) * c - l2s;
    float sum = wave_sum(q > 0.0f ? q * (l2q - l2p) : (q == 0.0f ? 0.0f : q));
    const float rest_m = no_rest ? 0.0f : rest.m;
    const float rest_l2 = no_rest ? 0.0f : log2_hw(rest.s);
    const float l2P = (rest_m - m) * c + rest_l2 - l2s;
    if (r > 0.0f) sum += r * (log2_hw(r) - l2P);
    const bool on = any_in && !empty;
    if (lane == 0) {
        if (loss) loss[row] = on ? sum * kLn2 : 0.0f;
        const float P = no_rest ? 0.0f : exp2_hw(l2P);
        stats[row] = DistillStats{rest_m, rest_l2, on ? (Q + r) * P - r : 0.0f, Q + r, m, l2s, norm,
                                  on ? 1.0f : 0.0f};
    }
}

// ---- gradients ----------------------------------------------------------------

// grad_j = p_j (A + B d_j) with d_j = log2 p_j, plus gl / T at the given token.
template <int kType, bool kEntropy>
__global__ __launch_bounds__(kBlock) void logprob_grad_kernel(
    const typename Elem<kType>::T* logits, int64_t vocab, int64_t stride, int32_t nchunk, float c,
    float inv_t, const int64_t* targets, const ProbStats* stats, const float* grad_logprob,
    const float* grad_entropy, typename Elem<kType>::T* grad, int64_t grad_stride) {
    constexpr int E = Elem<kType>::kE;
    const int64_t row = blockIdx.x / nchunk;
    const int64_t chunk = blockIdx.x % nchunk;
    const typename Elem<kType>::T* x = logits + row * stride;
    typename Elem<kType>::T* g = grad + row * grad_stride;
    const int64_t v0 = chunk * kChunkVecs + threadIdx.x;
    u32x4 r[kVecs];
    load_chunk<kType>(x, vocab, v0, r);
    const ProbStats st = stats[row];
    const int64_t t = targets ? targets[row] : -1;
    const bool given = t >= 0 && t < vocab;
    const float gl = given && grad_logprob && st.on != 0.0f ? grad_logprob[row] * inv_t : 0.0f;
    const float gh = kEntropy ? grad_entropy[row] * inv_t : 0.0f;
    const float A = -gl - gh * st.entropy, B = -gh * kLn2;
    const bool mine = given && t / kChunk<kType> == chunk && threadIdx.x == 0;
    const float xt = mine ? Elem<kType>::up(x[t]) : 0.0f;
    if (given) __syncthreads();                  // read before a gradient that replaces it is written
    auto value = [&](float v) {
        const float d = (v - st.m) * c - st.l2s;
        const float p = exp2_hw(d);
        return p * (kEntropy ? __builtin_fmaf(B, fmaxf(d, -200.0f), A) : A);
    };
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = value(Elem<kType>::get(r[i], e));
        store_vec<kType>(g, v0 + i * kBlock, vocab, pack<kType>(o));
    }
    if (given) {
        __syncthreads();                         // after the dense pass's write of the same entry
        if (mine) g[t] = Elem<kType>::down(value(xt) + gl);
    }
}

template <int kType>
__global__ __launch_bounds__(kBlock) void distill_grad_kernel(
    const typename Elem<kType>::T* logits, int64_t vocab, int64_t stride, int32_t nchunk, float c,
    float inv_t, const int64_t* ids, const float* tlp, int top, const DistillStats* stats,
    const float* grad_loss, typename Elem<kType>::T* grad, int64_t grad_stride) {
    constexpr int E = Elem<kType>::kE;
    const int64_t row = blockIdx.x / nchunk;
    const int64_t chunk = blockIdx.x % nchunk;
    const typename Elem<kType>::T* x = logits + row * stride;
    typename Elem<kType>::T* g = grad + row * grad_stride;
    const int64_t v0 = chunk * kChunkVecs + threadIdx.x;
    u32x4 r[kVecs];
    load_chunk<kType>(x, vocab, v0, r);
    const DistillStats st = stats[row];
    const float w = st.on != 0.0f ? grad_loss[row] * inv_t : 0.0f;
    // wave 0 forms the listed entries' gradients before any gradient is written
    int64_t id = -1;
    float listed = 0.0f;
    if (threadIdx.x < kWave) {
        const int lane = threadIdx.x;
        id = lane < top ? ids[row * top + lane] : -1;
        const bool in = id >= 0 && id < vocab;
        const float q = in ? exp2_hw(tlp[row * top + lane] * kLog2e - st.norm) : 0.0f;
        float sum = 0.0f;
        for (int k = 0; k < top; ++k) {
            const int64_t other = __shfl((long long)id, k);
            const float oq = __shfl(q, k);
            if (other == id) sum += oq;
        }
        if (!in || id / kChunk<kType> != chunk) id = -1;
        if (id >= 0) {
            const float p = exp2_hw((Elem<kType>::up(x[id]) - st.m) * c - st.l2s);
            listed = st.on != 0.0f ? w * (st.qr * p - sum) : 0.0f;
        }
    }
    __syncthreads();
    const float a = w * st.coef;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = a * exp2_hw((Elem<kType>::get(r[i], e) - st.rest_m) * c - st.rest_l2);
        store_vec<kType>(g, v0 + i * kBlock, vocab, pack<kType>(o));
    }
    __syncthreads();
    if (id >= 0) g[id] = Elem<kType>::down(listed);
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
    if (!workspace && need) return FLASHOPT_ERR_NULL;
    if (have < need || !aligned(workspace, 256)) return FLASHOPT_ERR_WORKSPACE;
    return FLASHOPT_OK;
}

static int check_list(const int64_t* top_id, const float* top_logprob, int32_t top, int64_t vocab) {
    if (top < 1 || top > FLASHOPT_TOP_MAX || top > vocab) return FLASHOPT_ERR_ARG;
    if (!top_id || !top_logprob) return FLASHOPT_ERR_NULL;
    if (!aligned(top_id, 8) || !aligned(top_logprob, 4)) return FLASHOPT_ERR_ALIGN;
    return FLASHOPT_OK;
}

static size_t parts_bytes(int32_t type, int64_t rows, int64_t vocab) {
    const size_t b = (size_t)(rows * chunks_of(type, vocab)) * sizeof(Part);
    return (b + 255) & ~size_t(255);
}

static float scale_of(double temperature) {
    return (float)(1.4426950408889634073599 / temperature);
}

// f is called with the type as a compile-time constant
template <typename F>
static int by_type(int32_t type, F f) {
    if (type == FLASHOPT_BF16) f(std::integral_constant<int, FLASHOPT_BF16>());
    else if (type == FLASHOPT_FP16) f(std::integral_constant<int, FLASHOPT_FP16>());
    else f(std::integral_constant<int, FLASHOPT_FP32>());
    return launch_status();
}

static void launch_logprob(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                           int64_t stride, double temperature, const int64_t* targets, int32_t top,
                           void* workspace, float* logprob, float* entropy, float* stats,
                           float* top_logprob, int64_t* top_id, hipStream_t st) {
    const int32_t nchunk = (int32_t)chunks_of(type, vocab);
    Part* part = (Part*)workspace;
    uint64_t* lists = (uint64_t*)((char*)workspace + parts_bytes(type, rows, vocab));
    const float c = scale_of(temperature);
    by_type(type, [&](auto k) {
        constexpr int kType = decltype(k)::value;
        const auto* x = (const typename Elem<kType>::T*)logits;
        const dim3 grid((unsigned)(rows * nchunk));
        if (top > 0)
            hipLaunchKernelGGL((chunk_kernel<kType, false, true>), grid, dim3(kBlock), 0, st, x,
                               vocab, stride, nchunk, c, nullptr, top, part, lists);
        else
            hipLaunchKernelGGL((chunk_kernel<kType, false, false>), grid, dim3(kBlock), 0, st, x,
                               vocab, stride, nchunk, c, nullptr, 0, part, lists);
        hipLaunchKernelGGL((logprob_join_kernel<kType>),
                           dim3((unsigned)((rows + kWavesPerBlock - 1) / kWavesPerBlock)),
                           dim3(kBlock), 0, st, x, rows, vocab, stride, nchunk, c, targets, top,
                           part, lists, logprob, entropy, (ProbStats*)stats, top_logprob, top_id);
    });
}

static int launch_logprob_grad(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                               int64_t stride, double temperature, const int64_t* targets,
                               const float* stats, const float* grad_logprob,
                               const float* grad_entropy, void* grad, int64_t grad_stride,
                               hipStream_t st) {
    const int32_t nchunk = (int32_t)chunks_of(type, vocab);
    const float c = scale_of(temperature), inv_t = (float)(1.0 / temperature);
    return by_type(type, [&](auto k) {
        constexpr int kType = decltype(k)::value;
        typedef typename Elem<kType>::T T;
        const dim3 grid((unsigned)(rows * nchunk));
        if (grad_entropy)
            hipLaunchKernelGGL((logprob_grad_kernel<kType, true>), grid, dim3(kBlock), 0, st,
                               (const T*)logits, vocab, stride, nchunk, c, inv_t, targets,
                               (const ProbStats*)stats, grad_logprob, grad_entropy, (T*)grad,
                               grad_stride);
        else
            hipLaunchKernelGGL((logprob_grad_kernel<kType, false>), grid, dim3(kBlock), 0, st,
                               (const T*)logits, vocab, stride, nchunk, c, inv_t, targets,
                               (const ProbStats*)stats, grad_logprob, grad_entropy, (T*)grad,
                               grad_stride);
    });
}

static void launch_distill(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                           int64_t stride, double temperature, const int64_t* top_id,
                           const float* top_logprob, int32_t top, int32_t tail, void* workspace,
                           float* loss, float* stats, hipStream_t st) {
    const int32_t nchunk = (int32_t)chunks_of(type, vocab);
    Part* part = (Part*)workspace;
    const float c = scale_of(temperature);
    by_type(type, [&](auto k) {
        constexpr int kType = decltype(k)::value;
        const auto* x = (const typename Elem<kType>::T*)logits;
        hipLaunchKernelGGL((chunk_kernel<kType, true, false>), dim3((unsigned)(rows * nchunk)),
                           dim3(kBlock), 0, st, x, vocab, stride, nchunk, c, top_id, top, part,
                           nullptr);
        hipLaunchKernelGGL((distill_join_kernel<kType>),
                           dim3((unsigned)((rows + kWavesPerBlock - 1) / kWavesPerBlock)),
                           dim3(kBlock), 0, st, x, rows, vocab, stride, nchunk, c, top_id,
                           top_logprob, top, tail, part, loss, (DistillStats*)stats);
    });
}

static int launch_distill_grad(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                               int64_t stride, double temperature, const int64_t* top_id,
                               const float* top_logprob, int32_t top, const float* stats,
                               const float* grad_loss, void* grad, int64_t grad_stride,
                               hipStream_t st) {
    const int32_t nchunk = (int32_t)chunks_of(type, vocab);
    const float c = scale_of(temperature), inv_t = (float)(1.0 / temperature);
    return by_type(type, [&](auto k) {
        constexpr int kType = decltype(k)::value;
        typedef typename Elem<kType>::T T;
        hipLaunchKernelGGL((distill_grad_kernel<kType>), dim3((unsigned)(rows * nchunk)),
                           dim3(kBlock), 0, st, (const T*)logits, vocab, stride, nchunk, c, inv_t,
                           top_id, top_logprob, top, (const DistillStats*)stats, grad_loss,
                           (T*)grad, grad_stride);
    });
}

}  // namespace flashopt

using namespace flashopt;

extern "C" {

size_t flashopt_logprob_workspace_bytes(int32_t type, int64_t rows, int64_t vocab, int32_t top) {
    if (!valid_type(type) || rows < 0 || vocab < 1 || vocab > FLASHOPT_VOCAB_MAX || top < 0 ||
        top > FLASHOPT_TOP_MAX || rows > INT32_MAX / ((vocab + 4095) / 4096))
        return 0;
    return parts_bytes(type, rows, vocab) +
           (size_t)(rows * chunks_of(type, vocab)) * (size_t)top * sizeof(uint64_t);
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
    launch_logprob(logits, type, rows, vocab, stride, temperature, targets, top, workspace,
                   logprob, entropy, stats, top_logprob, top_id, (hipStream_t)stream);
    return launch_status();
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
    return launch_logprob_grad(logits, type, rows, vocab, stride, temperature, targets, stats,
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
    launch_logprob(logits, type, rows, vocab, stride, temperature, targets, 0, workspace, logprob,
                   entropy, stats, nullptr, nullptr, (hipStream_t)stream);
    return launch_logprob_grad(logits, type, rows, vocab, stride, temperature, targets, stats,
                               grad_logprob, grad_entropy, grad, grad_stride, (hipStream_t)stream);
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
    launch_distill(logits, type, rows, vocab, stride, temperature, top_id, top_logprob, top, tail,
                   workspace, loss, stats, (hipStream_t)stream);
    return launch_status();
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
    return launch_distill_grad(logits, type, rows, vocab, stride, temperature, top_id, top_logprob,
                               top, stats, grad_loss, grad, grad_stride, (hipStream_t)stream);
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
    launch_distill(logits, type, rows, vocab, stride, temperature, top_id, top_logprob, top, tail,
                   workspace, loss, stats, (hipStream_t)stream);
    return launch_distill_grad(logits, type, rows, vocab, stride, temperature, top_id, top_logprob,
                               top, stats, grad_loss, grad, grad_stride, (hipStream_t)stream);
}

}  // extern "C"
