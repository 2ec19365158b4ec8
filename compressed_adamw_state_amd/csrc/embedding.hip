// Rows of an embedding table for given tokens, and the table's gradient
// (include/flashopt_lm.h).
//
// grad[v] = scale * sum of dy[i] over the i with ids[i] = v.  The positions i are put in
// the order of their ids, equal ids by position, so that a token's rows of dy stand
// together and are added in that order whatever the launch: no atomic adds to
// memory, the same bits every time.
//
//   sort    a block takes every 256th id (common ones, which stand together in a
//           vocabulary, go to blocks of their own; the order is of the blocks, then the
//           ids).  Each of its waves goes over its own part of the positions: it
//           counts and lists the block's ids among them, and (with what the other waves
//           and the blocks before it have counted) puts each position into its place;
//           lanes with equal ids rank by lane.
//   sums    a block takes kept positions in their order, a piece of them and a
//           slice of the columns.  A token that lies in one piece is written at
//           once, the parts of one that does not go to the workspace.  Other
//           blocks of the launch write the zeros of the tokens that no id names.
//   join    the parts of a token added in order.
//
// 16384 positions, 128256 x 4096 BF16: 238 to 256 us (by the card), of which the sums' launch,
// 1.2 GB written and read, takes 218 to 236 (sort 12, join 9); 2047 positions, 50257 x 768
// FP32: 35 (8, 23, 4).  Every block reads all ids, so sorting grows with 256 (512) n whatever
// the columns: 65536 of them 27 us, 16 MB from each L2, beside sums of 41 us for 1024 BF16 columns and
// 27 for 64; 2^20 of them 1057 beside 462 and 357.
#include <cmath>

#include "rows.hpp"

namespace flashopt {

// ---- lookup ------------------------------------------------------------------------

constexpr int kLookupWords = 4;

// from: weight rows of the output's type (int8_t: codes with a scale a row)
template <int kType, typename From>
__global__ __launch_bounds__(kBlock) void lookup_kernel(const int64_t* ids, int64_t n,
                                                        const From* weight, const float* w_scale,
                                                        int64_t vocab, int64_t dim,
                                                        int64_t weight_stride, float scale,
                                                        typename Elem<kType>::T* out,
                                                        int64_t out_stride, uint32_t words) {
    constexpr int E = Elem<kType>::kE;
    constexpr bool kCodes = sizeof(From) == 1;
    constexpr int64_t kStep = kLookupWords * kBlock;
    const int64_t total = n * words;
    for (int64_t first = blockIdx.x * kStep; first < total; first += gridDim.x * kStep) {
        const int64_t row0 = first / words;
        const uint32_t w0 = (uint32_t)(first - row0 * words);
        int64_t row[kLookupWords], id[kLookupWords];
        uint32_t word[kLookupWords];
#pragma unroll
        for (int i = 0; i < kLookupWords; ++i) {
            const uint32_t w = w0 + i * kBlock + threadIdx.x;
            row[i] = row0 + w / words;
            word[i] = w % words;
            id[i] = row[i] < n ? ids[row[i]] : -1;
        }
        u32x4 v[kLookupWords];
        float s[kLookupWords];
        bool in[kLookupWords];
#pragma unroll
        for (int i = 0; i < kLookupWords; ++i) {
            in[i] = id[i] >= 0 && id[i] < vocab;
            if (!in[i]) id[i] = 0;               // read, not used
            s[i] = in[i] ? scale : 0.0f;
        }
        if constexpr (kCodes) {                  // rows are padded to 128 codes
#pragma unroll
            for (int i = 0; i < kLookupWords; ++i) {
                const uint32_t* c = reinterpret_cast<const uint32_t*>(weight + id[i] * weight_stride + (int64_t)word[i] * E);
                v[i][0] = c[0];
                if (E == 8) v[i][1] = c[1];
                s[i] *= w_scale[id[i]];
            }
        } else {
            load_words<kType>(v, dim, dim % E == 0, [&](int i) { return WordAt<kType>{weight + id[i] * weight_stride, word[i]}; });
        }
#pragma unroll
        for (int i = 0; i < kLookupWords; ++i) {
            if (row[i] >= n) continue;
            float x[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if constexpr (kCodes) x[e] = (float)(int8_t)(v[i][e / 4] >> (8 * (e % 4))) * s[i];
                else x[e] = Elem<kType>::get(v[i], e) * s[i];
                if (!in[i]) x[e] = 0.0f;
            }
            store_vec<kType>(out + row[i] * out_stride, word[i], dim, pack<kType>(x));
        }
    }
}

// ---- the positions in the order of their ids -------------------------------------------

constexpr int kSortWaves = 16, kSortThreads = kSortWaves * kWave;
constexpr int kRunMost = 1024;                   // ids of a block: one a thread

// A kept position, its id, and where that id's positions begin and end in their order
// (together, so that one load tells all that the sums need).
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
struct Sorted {
    int32_t* start;                              // by place(id), and the end of the last
    i32x4* at;                                   // in that order
    int32_t run, shift;                          // ids of a block, of 2^shift blocks
    __device__ __forceinline__ int32_t place(int32_t id) const {
        return (id & ((1 << shift) - 1)) * run + (id >> shift);
    }
    __device__ __forceinline__ int32_t kept() const { return start[run << shift]; }
};

// A wave's found positions, in LDS: the position, from the wave's first on, and id / blocks in one
// word, of 22 and 10 bits.  A wave that finds more goes over its positions again instead.
constexpr int kFound = 512;
static_assert(FLASHOPT_EMBED_MAX / kSortWaves < 1 << 22 && kRunMost <= 1 << 10 &&
              FLASHOPT_VOCAB_MAX <= 512 * kRunMost, "both fit");

__global__ __launch_bounds__(kSortThreads) void sort_kernel(const int64_t* ids, int32_t n,
                                                            int32_t vocab, int bits, Sorted to) {
    extern __shared__ int32_t count[];           // [kSortWaves][run], then [run + 1] starts
    __shared__ uint32_t list[kSortWaves][kFound];
    __shared__ int32_t below[kSortWaves], sums[kSortWaves];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int run = to.run, shift = to.shift;
    const uint32_t block = blockIdx.x, low_bits = (1u << shift) - 1;
    for (int i = tid; i < kSortWaves * run; i += kSortThreads) count[i] = 0;
    __syncthreads();
    int32_t* mine = count + wave * run;
    // this wave's positions
    const int32_t part = ((n + kSortWaves - 1) / kSortWaves + kWave - 1) / kWave * kWave;
    const int32_t begin = min(wave * part, n), end = min(begin + part, n);
    constexpr int U = 16;                        // loads on their way at a time
    // f(position, whether it has an id, the id)
    auto each = [&](auto f) {
        for (int32_t i = begin; i < end; i += U * kWave) {
            int64_t id[U];
#pragma unroll
            for (int u = 0; u < U; ++u) id[u] = ids[min(i + u * kWave + lane, end - 1)];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i + u * kWave >= end) break;
                const int32_t p = i + u * kWave + lane;
                const bool in = p < end && id[u] >= 0 && id[u] < vocab;
                f(p, in, (uint32_t)id[u]);
            }
        }
    };
    int32_t lower = 0, found = 0;
    each([&](int32_t p, bool in, uint32_t id) {
        lower += __popcll(__ballot(in && (id & low_bits) < block));
        const bool here = in && (id & low_bits) == block;
        const uint64_t who = __ballot(here);
        if (who == 0) return;                    // most often
        if (here) {
            const uint32_t k = id >> shift;
            const int32_t at = found + __popcll(who & ((uint64_t(1) << lane) - 1));
            if (at < kFound) list[wave][at] = (uint32_t)(p - begin) << 10 | k;
            atomicAdd(&mine[k], 1);
        }
        found += __popcll(who);
    });
    if (lane == 0) below[wave] = lower;
    __syncthreads();
    // a thread an id: where its positions begin, and those of each wave
    int32_t total = 0, base = 0;
    for (int w = 0; w < kSortWaves; ++w) {
        base += below[w];
        if (tid < run) total += count[w * run + tid];
    }
    int32_t scan = total;                        // of the threads up to this one
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int32_t x = __shfl_up(scan, o);
        if (lane >= o) scan += x;
    }
    if (lane == kWave - 1) sums[wave] = scan;
    __syncthreads();
    int32_t from = base + scan - total;
    for (int w = 0; w < wave; ++w) from += sums[w];
    int32_t* start = count + kSortWaves * run;
    if (tid < run) {
        start[tid] = from;
        if (tid == run - 1) start[run] = from + total;
        to.start[block * run + tid] = from;
        if (tid == run - 1 && block == gridDim.x - 1) to.start[gridDim.x * run] = from + total;
        for (int w = 0; w < kSortWaves; ++w) {
            const int32_t c = count[w * run + tid];
            count[w * run + tid] = from;
            from += c;
        }
    }
    __syncthreads();
    volatile int32_t* next = mine;               // only this wave's, in its order
    auto place = [&](int32_t p, uint32_t k, bool in) {
        uint64_t same = __ballot(in);
        if (same == 0) return;
        if (!in) k = 0;
        for (int b = 0; b < bits; ++b) {
            const bool bit = (k >> b) & 1;
            const uint64_t with = __ballot(bit);
            same &= bit ? with : ~with;
        }
        if (in) {
            const int32_t at = next[k];
            to.at[at + __popcll(same & ((uint64_t(1) << lane) - 1))] = i32x4{p, (int32_t)(k << shift | block), start[k], start[k + 1]};
            if ((same >> lane) == 1) next[k] = at + __popcll(same);           // the last of them
        }
    };
    if (found <= kFound) {
        for (int32_t i = 0; i < found; i += kWave) {
            const uint32_t e = i + lane < found ? list[wave][i + lane] : 0;
            place(begin + (int32_t)(e >> 10), e & 1023, i + lane < found);
        }
    } else {
        each([&](int32_t p, bool in, uint32_t id) { place(p, id >> shift, in && (id & low_bits) == block); });
    }
}

// ---- sums ---------------------------------------------------------------------------

constexpr int kAhead = 16;                       // rows of dy loaded before the first is added
constexpr int64_t kZeroWords = 4096;             // of zeros that a block writes

template <int kType>
struct TableGrad {
    typedef typename Elem<kType>::T T;
    const T* dy;
    int64_t dy_stride, dim;
    int32_t n, vocab, piece, pieces, slices, threads, zero_rows;
    float scale;
    bool beyond;                                 // a table that no cache holds
    Sorted in;
    float* part;                                 // pieces x 2 x dim
    T* grad;
    int64_t grad_stride;
};

template <int kType>
__global__ __launch_bounds__(kBlock) void sums_kernel(TableGrad<kType> a) {
    constexpr int E = Elem<kType>::kE;
    typedef typename Elem<kType>::T T;
    extern __shared__ int32_t held[];
    const int32_t tid = threadIdx.x;
    const uint32_t units = (uint32_t)a.pieces * a.slices;
    const int64_t words = (a.dim + E - 1) / E;
    if (blockIdx.x >= units) {                   // rows of zeros
        const int32_t v0 = (int32_t)(blockIdx.x - units) * a.zero_rows;
        const int32_t rows = min(a.zero_rows, a.vocab - v0);
        // all of the rows' starts at once, not one after the other
        if (tid < rows) {
            const int32_t p = a.in.place(v0 + tid);
            held[tid] = a.in.start[p] == a.in.start[p + 1];
        }
        __syncthreads();
        T* g = a.grad + v0 * a.grad_stride;
        int64_t w = tid;
        int32_t v = 0;
        const u32x4 zero = {0, 0, 0, 0};
        while (v < rows) {                       // all of the block's words in turn
            if (w >= words) {
                w -= words;
                ++v;
                continue;
            }
            T* row = g + v * a.grad_stride;
            if (held[v]) {
                if (a.beyond && w * E + E <= a.dim) __builtin_nontemporal_store(zero, reinterpret_cast<u32x4_any*>(row + w * E));
                else store_vec<kType>(row, w, a.dim, zero);
            }
            w += a.threads;
        }
        return;
    }
    // what follows a position's row: another of its token, or the token's sum is to be
    // written to the table, or, of one that other pieces share, as its last or first part
    enum { kMore = 0, kTable = 1, kLast = 2, kFirst = 3 };
    const int32_t c = (int32_t)(blockIdx.x / a.slices), first = c * a.piece;
    const int32_t kept = a.in.kept();
    int32_t *at = held, *id = held + a.piece, *then = id + a.piece;
    for (int32_t i = tid; i < a.piece; i += a.threads) {
        const i32x4 r = a.in.at[min(first + i, a.n - 1)];        // (behind the kept ones: not used)
        const int32_t stop = min(first + a.piece, kept);
        at[i] = r[0];
        id[i] = r[1];
        then[i] = first + i + 1 < min(r[3], stop) ? kMore
                  : r[2] >= first && r[3] <= stop ? kTable : r[2] < first ? kLast : kFirst;
    }
    const int32_t count = min(a.piece, kept - first);
    if (count <= 0) return;
    __syncthreads();
    const int64_t w = (int64_t)(blockIdx.x % a.slices) * a.threads + tid;
    const bool there = w < words;
    float sum[E] = {};
    for (int32_t i0 = 0; i0 < count; i0 += kAhead) {
        u32x4 v[kAhead];
        load_words<kType>(v, a.dim, a.dim % (E * a.threads) == 0, [&](int u) {
            return WordAt<kType>{a.dy + at[min(i0 + u, count - 1)] * a.dy_stride, w};
        });
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int32_t i = i0 + u;
            if (i >= count) break;
#pragma unroll
            for (int e = 0; e < E; ++e) sum[e] += Elem<kType>::get(v[u], e);
            const int32_t what = then[i];
            if (what == kMore) continue;
            if (what == kTable) {
                float x[E];
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = sum[e] * a.scale;
                if (there) store_vec<kType>(a.grad + id[i] * a.grad_stride, w, a.dim, pack<kType>(x));
            } else if (there) {
                uint32_t* p = (uint32_t*)a.part + (2 * (int64_t)c + (what == kLast ? 0 : 1)) * a.dim;
#pragma unroll
                for (int h = 0; h < E / 4; ++h)
                    store_vec<FLASHOPT_FP32>(p, w * (E / 4) + h, a.dim, u32x4{as_u32(sum[4 * h]), as_u32(sum[4 * h + 1]), as_u32(sum[4 * h + 2]), as_u32(sum[4 * h + 3])});
            }
#pragma unroll
            for (int e = 0; e < E; ++e) sum[e] = 0.0f;
        }
    }
}

// The token that begins in piece c and goes beyond it, if there is one.
template <int kType>
__global__ __launch_bounds__(kBlock) void join_kernel(TableGrad<kType> a) {
    constexpr int E = Elem<kType>::kE;
    const int32_t c = (int32_t)(blockIdx.x / a.slices), next = (c + 1) * a.piece;
    if (next >= a.in.kept()) return;
    const i32x4 r = a.in.at[next - 1];
    const int32_t id = r[1], begin = r[2], end = r[3];
    if (begin < c * a.piece || end <= next) return;
    const int64_t w = (int64_t)(blockIdx.x % a.slices) * a.threads + threadIdx.x;
    if (w * E >= a.dim) return;
    const int32_t last = (end - 1) / a.piece;
    // (a thread's E columns are whole words of the parts, up to the row's end)
    constexpr int H = E / 4, kParts = 16;
    const uint32_t* part = (const uint32_t*)a.part;
    const bool whole = a.dim % 4 == 0 && (w + 1) * E <= a.dim;
    float x[E];
    u32x4 one[H];
    load_words<FLASHOPT_FP32>(one, a.dim, whole, [&](int h) {
        return WordAt<FLASHOPT_FP32>{part + (2 * (int64_t)c + 1) * a.dim, w * H + h};
    });
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = as_f32(one[e / 4][e % 4]);
    for (int32_t d = c + 1; d <= last; d += kParts) {
        u32x4 v[kParts * H];
        load_words<FLASHOPT_FP32>(v, a.dim, whole, [&](int i) {
            return WordAt<FLASHOPT_FP32>{part + 2 * (int64_t)min(d + i / H, last) * a.dim, w * H + i % H};
        });
#pragma unroll
        for (int u = 0; u < kParts; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = d + u <= last ? x[e] + as_f32(v[u * H + e / 4][e % 4]) : x[e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= a.scale;
    store_vec<kType>(a.grad + id * a.grad_stride, w, a.dim, pack<kType>(x));
}

// ---- host ---------------------------------------------------------------------

template <typename F>
static int by_type(int32_t type, F f) {
    if (type == FLASHOPT_BF16) f(std::integral_constant<int, FLASHOPT_BF16>());
    else if (type == FLASHOPT_FP16) f(std::integral_constant<int, FLASHOPT_FP16>());
    else f(std::integral_constant<int, FLASHOPT_FP32>());
    return launch_status();
}

static int check_table(int32_t type, int64_t n, int64_t vocab, int64_t dim, double scale) {
    if (!valid_type(type)) return FLASHOPT_ERR_ARG;
    if (n < 0 || n > FLASHOPT_EMBED_MAX || vocab < 1 || vocab > FLASHOPT_VOCAB_MAX || dim < 1 ||
        dim > FLASHOPT_INT8_COLS_MAX)
        return FLASHOPT_ERR_SIZE;
    return std::isfinite((float)scale) ? FLASHOPT_OK : FLASHOPT_ERR_ARG;
}

// two spans of rows (strides and lengths in elements of the same size)
static bool spans_meet(size_t size, const void* a, int64_t a_rows, int64_t a_stride, const void* b,
                       int64_t b_rows, int64_t b_stride, int64_t cols) {
    const __int128 p = (uintptr_t)a, q = (uintptr_t)b;
    return p < q + ((__int128)(b_rows - 1) * b_stride + cols) * (__int128)size &&
           q < p + ((__int128)(a_rows - 1) * a_stride + cols) * (__int128)size;
}

// rows of `size` bytes an element, and a block of bytes
static bool block_meets(size_t size, const void* a, int64_t rows, int64_t stride, int64_t cols,
                        const void* b, int64_t bytes) {
    return rows_meet(rows, a, (__int128)stride * (int64_t)size, cols * (int64_t)size, b, bytes);
}

static dim3 lookup_grid(int64_t total) {
    const int64_t blocks = (total + kLookupWords * kBlock - 1) / (kLookupWords * kBlock);
    return dim3((unsigned)(blocks < (int64_t(1) << 22) ? blocks : int64_t(1) << 22));
}

// Positions of a piece: few where they are few in all, so that a block has one round of
// loads; more from 4096 on, so that the parts of one token stay few.  Sums and join:
// 16384 positions, 128256 x 4096 BF16: 219 + 11 us with 32, 235 + 18 with 16; 65536 positions,
// 32000 x 1024: 33 + 18 with 32, 36 + 10 with 64, 49 + 7 with 128.
static int64_t piece_of(int64_t n) {
    int64_t p = 8;
    while (p < 2048 && p * (p < 32 ? 512 : 1024) < n) p *= 2;
    return p;
}

struct TablePlan {
    int32_t run, shift;
    int64_t piece, pieces;
    size_t start, at, part;                      // bytes
};
static TablePlan table_plan(int64_t n, int64_t vocab, int64_t dim) {
    auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
    TablePlan p;
    p.piece = piece_of(n);
    p.pieces = (n + p.piece - 1) / p.piece;
    // 256 blocks, a CU each, twice as many where their ids would be more than kRunMost
    p.shift = vocab <= 256 * kRunMost ? 8 : 9;
    p.run = (int32_t)((vocab + (1 << p.shift) - 1) >> p.shift);
    p.start = up((((size_t)p.run << p.shift) + 1) * 4);
    p.at = up((size_t)n * 16);
    p.part = up((size_t)p.pieces * 2 * dim * 4);
    return p;
}

}  // namespace flashopt

using namespace flashopt;

extern "C" {

int flashopt_embedding(const int64_t* ids, int64_t n, const void* weight, int32_t type,
                       int64_t vocab, int64_t dim, int64_t weight_stride, double scale, void* out,
                       int64_t out_stride, void* stream) {
    const int e = check_table(type, n, vocab, dim, scale);
    if (e) return e;
    if (weight_stride < dim || weight_stride > kMaxNumel || out_stride < dim || out_stride > kMaxNumel)
        return FLASHOPT_ERR_SIZE;
    if (n == 0) return FLASHOPT_OK;
    if (!ids || !weight || !out) return FLASHOPT_ERR_NULL;
    const size_t size = type_size(type);
    if (!aligned(ids, 8) || !aligned(weight, size) || !aligned(out, size)) return FLASHOPT_ERR_ALIGN;
    if (spans_meet(size, weight, vocab, weight_stride, out, n, out_stride, dim) ||
        block_meets(size, out, n, out_stride, dim, ids, n * 8))
        return FLASHOPT_ERR_ARG;
    return by_type(type, [&](auto t) {
        constexpr int kType = decltype(t)::value;
        typedef typename Elem<kType>::T T;
        const uint32_t words = (uint32_t)((dim + Elem<kType>::kE - 1) / Elem<kType>::kE);
        hipLaunchKernelGGL((lookup_kernel<kType, T>), lookup_grid(n * words), dim3(kBlock), 0,
                           (hipStream_t)stream, ids, n, (const T*)weight, nullptr, vocab, dim,
                           weight_stride, (float)scale, (T*)out, out_stride, words);
    });
}

int flashopt_embedding_int8(const int64_t* ids, int64_t n, const int8_t* w, const float* w_scale,
                            int64_t vocab, int64_t dim, double scale, void* out, int32_t type,
                            int64_t out_stride, void* stream) {
    const int e = check_table(type, n, vocab, dim, scale);
    if (e) return e;
    if (out_stride < dim || out_stride > kMaxNumel) return FLASHOPT_ERR_SIZE;
    if (n == 0) return FLASHOPT_OK;
    if (!ids || !w || !w_scale || !out) return FLASHOPT_ERR_NULL;
    if (!aligned(ids, 8) || !aligned(w, 16) || !aligned(w_scale, 4) || !aligned(out, type_size(type)))
        return FLASHOPT_ERR_ALIGN;
    const size_t size = type_size(type);
    if (block_meets(size, out, n, out_stride, dim, w, vocab * flashopt_int8_ld(dim)) ||
        block_meets(size, out, n, out_stride, dim, w_scale, vocab * 4) ||
        block_meets(size, out, n, out_stride, dim, ids, n * 8))
        return FLASHOPT_ERR_ARG;
    return by_type(type, [&](auto t) {
        constexpr int kType = decltype(t)::value;
        typedef typename Elem<kType>::T T;
        const uint32_t words = (uint32_t)((dim + Elem<kType>::kE - 1) / Elem<kType>::kE);
        hipLaunchKernelGGL((lookup_kernel<kType, int8_t>), lookup_grid(n * words), dim3(kBlock), 0,
                           (hipStream_t)stream, ids, n, w, w_scale, vocab, dim,
                           flashopt_int8_ld(dim), (float)scale, (T*)out, out_stride, words);
    });
}

size_t flashopt_embedding_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
    if (check_table(FLASHOPT_BF16, n, vocab, dim, 1.0)) return 0;
    const TablePlan p = table_plan(n, vocab, dim);
    return p.start + p.at + p.part;
}

int flashopt_embedding_backward(const int64_t* ids, int64_t n, const void* dy, int32_t type,
                                int64_t dy_stride, int64_t vocab, int64_t dim, double scale,
                                void* workspace, size_t workspace_bytes, void* grad,
                                int64_t grad_stride, void* stream) {
    const int e = check_table(type, n, vocab, dim, scale);
    if (e) return e;
    if (dy_stride < dim || dy_stride > kMaxNumel || grad_stride < dim || grad_stride > kMaxNumel)
        return FLASHOPT_ERR_SIZE;
    if (!grad || !workspace || (n > 0 && (!ids || !dy))) return FLASHOPT_ERR_NULL;
    const size_t size = type_size(type);
    if (!aligned(ids, 8) || !aligned(dy, size) || !aligned(grad, size)) return FLASHOPT_ERR_ALIGN;
    const TablePlan p = table_plan(n, vocab, dim);
    if (workspace_bytes < p.start + p.at + p.part || !aligned(workspace, 256)) return FLASHOPT_ERR_WORKSPACE;
    if (n > 0 && (spans_meet(size, dy, n, dy_stride, grad, vocab, grad_stride, dim) ||
                  block_meets(size, grad, vocab, grad_stride, dim, ids, n * 8)))
        return FLASHOPT_ERR_ARG;
    const hipStream_t st = (hipStream_t)stream;
    char* ws = (char*)workspace;
    const Sorted sorted = {(int32_t*)ws, (i32x4*)(ws + p.start), p.run, p.shift};
    int bits = 0;
    while ((1 << bits) < sorted.run) ++bits;
    hipLaunchKernelGGL(sort_kernel, dim3(1u << sorted.shift), dim3(kSortThreads),
                       (size_t)(sorted.run * (kSortWaves + 1) + 1) * 4, st, ids, (int32_t)n,
                       (int32_t)vocab, bits, sorted);
    return by_type(type, [&](auto t) {
        constexpr int kType = decltype(t)::value;
        typedef typename Elem<kType>::T T;
        const int64_t words = (dim + Elem<kType>::kE - 1) / Elem<kType>::kE;
        TableGrad<kType> a = {};
        a.dy = (const T*)dy;
        a.dy_stride = dy_stride;
        a.dim = dim;
        a.n = (int32_t)n;
        a.vocab = (int32_t)vocab;
        a.piece = (int32_t)p.piece;
        a.pieces = (int32_t)p.pieces;
        a.threads = (int32_t)(words < kBlock ? (words + kWave - 1) / kWave * kWave : kBlock);
        a.slices = (int32_t)((words + a.threads - 1) / a.threads);
        // rows of zeros: kZeroWords a block, fewer where there would be less than four blocks a CU
        int64_t rows = words < kZeroWords ? (kZeroWords + words - 1) / words : 1;
        if (rows > (vocab + 1023) / 1024) rows = (vocab + 1023) / 1024;
        if (rows > a.threads) rows = a.threads;
        a.zero_rows = (int32_t)rows;
        a.scale = (float)scale;
        // Non-temporal zeros: a table of 128256 x 4096 in BF16 232 us for 252, but one of 50257 x
        // 768, which the last-level cache holds, in FP32 42 for 34, in BF16 27 for 22.
        a.beyond = (double)vocab * (double)dim * (double)size > 256e6;
        a.in = sorted;
        a.part = (float*)(ws + p.start + p.at);
        a.grad = (T*)grad;
        a.grad_stride = grad_stride;
        const int64_t zero = (vocab + a.zero_rows - 1) / a.zero_rows;
        const unsigned units = (unsigned)(p.pieces * a.slices);
        hipLaunchKernelGGL((sums_kernel<kType>), dim3(units + (unsigned)zero), dim3(a.threads),
                           (size_t)(p.piece * 12 > a.threads * 4 ? p.piece * 12 : a.threads * 4), st, a);
        if (p.pieces > 1)
            hipLaunchKernelGGL((join_kernel<kType>), dim3((unsigned)((p.pieces - 1) * a.slices)),
                               dim3(a.threads), 0, st, a);
    });
}

}  // extern "C"
