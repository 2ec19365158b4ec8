// Losses of log probabilities (include/flashopt_lm.h): the policy loss token by
// token, and preferences over pairs of sequences.
//
// A pair's loss needs its two sums before any of its gradients.  One block takes
// a pair, sums its tokens and writes their gradients; where there are few pairs of
// many tokens, several blocks share a pair in two launches, each of which forms
// the pair's sums from all of its blocks' parts, in their order.  Sums are
// binary64: the reward is a small difference of long sums, and a token costs one
// addition beside its 12 bytes.  300 pairs of 0 to 1500 tokens a sequence: 7 us forward and
// 7 backward, latency of a pair's loads, sums over the block and exponentials.
#include <cmath>

#include "policy.hpp"

namespace flashopt {

// ---- policy ------------------------------------------------------------------------

__global__ __launch_bounds__(kBlock) void policy_kernel(const float* logprob, PolicyIn in,
                                                        const uint8_t* mask, int64_t n,
                                                        const float* grad_loss, float* grad) {
    for (int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x; i < n; i += (int64_t)gridDim.x * kBlock) {
        const float w = in.weight ? in.weight[i] : 1.0f;
        PolicyRow r = {0.0f, 0.0f, 0.0f};
        if (w != 0.0f && !(mask && mask[i] == 0)) {
            r = policy_row(logprob[i], 0.0f, in, i, w);
            if (grad_loss) r.gl *= grad_loss[i];
        }
        if (in.loss) in.loss[i] = r.loss;
        if (grad) grad[i] = r.gl;
    }
}

// ---- preferences ---------------------------------------------------------------

constexpr int kPairThreads = 512, kPairWaves = kPairThreads / kWave;

struct PairSums {
    double sum[2], count[2];                     // chosen, rejected
};

__device__ __forceinline__ double wave_total(double x) {
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) x += __shfl_xor(x, o);
    return x;
}

__device__ __forceinline__ bool counted(const PreferenceIn& in, int64_t t) {
    if (in.mask && in.mask[t] == 0) return false;
    return !in.targets || (in.targets[t] >= 0 && in.targets[t] < in.vocab);
}

// offset i, where it may be used
__device__ __forceinline__ int64_t offset_of(const PreferenceIn& in, int64_t i) {
    const int64_t o = in.offsets[i];
    return o < 0 ? 0 : o > in.tokens ? in.tokens : o;
}

// this block's share of a pair: every `shares`-th run of kPairThreads tokens
template <typename F>
__device__ __forceinline__ void each_token(int64_t begin, int64_t end, int share, int shares, F f) {
    for (int64_t t = begin + (int64_t)share * kPairThreads + threadIdx.x; t < end; t += (int64_t)shares * kPairThreads) f(t);
}

// Every thread gets the block's sums.
__device__ __forceinline__ PairSums block_sums(const PreferenceIn& in, const int64_t* at, int share,
                                               int shares, double (*red)[4]) {
    double s[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int side = 0; side < 2; ++side)
        each_token(at[side], at[side + 1], share, shares, [&](int64_t t) {
            if (!counted(in, t)) return;
            s[side] += in.ref ? (double)in.logprob[t] - (double)in.ref[t] : (double)in.logprob[t];
            s[2 + side] += 1.0;
        });
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        s[k] = wave_total(s[k]);
        if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave][k] = s[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        s[k] = 0.0;
        for (int w = 0; w < kPairWaves; ++w) s[k] += red[w][k];
    }
    return PairSums{{s[0], s[1]}, {s[2], s[3]}};
}

// The parts of a pair's blocks in their order.
__device__ __forceinline__ PairSums join_sums(const PairSums* parts, int shares) {
    PairSums s = parts[0];
    for (int i = 1; i < shares; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            s.sum[k] += parts[i].sum[k];
            s.count[k] += parts[i].count[k];
        }
    return s;
}

// kStep 0: a block a pair, all of it; 1: the parts of the pairs' sums; 2: the rest
template <int kStep>
__global__ __launch_bounds__(kPairThreads) void preference_kernel(PreferenceIn in, int shares,
                                                                  PairSums* parts) {
    __shared__ double red[kPairWaves][4];
    const int64_t pair = blockIdx.x / (unsigned)shares;
    const int share = blockIdx.x % (unsigned)shares;
    int64_t at[3];
    at[0] = offset_of(in, 2 * pair);
    at[1] = max(at[0], offset_of(in, 2 * pair + 1));
    at[2] = max(at[1], offset_of(in, 2 * pair + 2));
    PairSums s;
    if (kStep == 2) {
        s = join_sums(parts + pair * shares, shares);
    } else {
        s = block_sums(in, at, share, shares, red);
        if (kStep == 1) {
            if (threadIdx.x == 0) parts[blockIdx.x] = s;
            return;
        }
    }
    double per[2], r[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        per[k] = in.average ? 1.0 / fmax(s.count[k], 1.0) : 1.0;
        r[k] = in.beta * s.sum[k] * per[k];
    }
    const double d = r[0] - r[1] - in.margin, e = exp(-fabs(d)), low = log1p(e);
    if (share == 0 && threadIdx.x == 0) {
        if (in.reward) {
            in.reward[2 * pair] = (float)r[0];
            in.reward[2 * pair + 1] = (float)r[1];
        }
        // log(1 + e^-d) = max(0, -d) + log(1 + e^-|d|), NaN where d is, and log(1 + e^d); one of
        // them is infinite where d is, and of weight 0 then not 0 * infinity
        if (in.loss) {
            double x = 0.0;
            if (in.smoothing < 1.0) x = (1.0 - in.smoothing) * ((d > 0.0 ? 0.0 : -d) + low);
            if (in.smoothing > 0.0) x += in.smoothing * ((d > 0.0 ? d : 0.0) + low);
            in.loss[pair] = (float)x;
        }
    }
    if (!in.grad) return;
    // 1 / (1 + e^d) and 1 / (1 + e^-d)
    const double small = e / (1.0 + e), large = 1.0 / (1.0 + e);
    const double minus = d > 0.0 ? small : large, plus = d > 0.0 ? large : small;
    const double slope = (in.smoothing * plus - (1.0 - in.smoothing) * minus) *
                         (in.grad_loss ? (double)in.grad_loss[pair] : 1.0) * in.beta;
    const float g[2] = {(float)(slope * per[0]), (float)(-slope * per[1])};
#pragma unroll
    for (int side = 0; side < 2; ++side)
        each_token(at[side], at[side + 1], share, shares,
                   [&](int64_t t) { in.grad[t] = counted(in, t) ? g[side] : 0.0f; });
    // tokens before the first sequence and behind the last
    const int64_t first = offset_of(in, 0), last = offset_of(in, 2 * in.pairs);
    const int64_t me = (int64_t)blockIdx.x * kPairThreads + threadIdx.x, step = (int64_t)gridDim.x * kPairThreads;
    for (int64_t t = me; t < first; t += step) in.grad[t] = 0.0f;
    for (int64_t t = max(first, last) + me; t < in.tokens; t += step) in.grad[t] = 0.0f;
}

// no pairs: every token is outside
__global__ __launch_bounds__(kBlock) void no_pairs_kernel(float* grad, int64_t tokens) {
    for (int64_t t = (int64_t)blockIdx.x * kBlock + threadIdx.x; t < tokens; t += (int64_t)gridDim.x * kBlock)
        grad[t] = 0.0f;
}

// ---- host ---------------------------------------------------------------------

// Blocks of a pair: until 512 run, of at least 2048 tokens each on average.
static int64_t shares_of(int64_t pairs, int64_t tokens) {
    if (pairs < 1) return 1;
    int64_t s = 512 / pairs, most = tokens / pairs / 2048;
    if (s > most) s = most;
    return s < 1 ? 1 : s > 32 ? 32 : s;
}

size_t preference_workspace(int64_t pairs, int64_t tokens) {
    const int64_t s = shares_of(pairs, tokens);
    return s == 1 ? 0 : ((size_t)(pairs * s) * sizeof(PairSums) + 255) & ~size_t(255);
}

int check_preference(int64_t pairs, int64_t tokens, double beta, double margin, double smoothing,
                     int32_t average) {
    if (pairs < 0 || pairs > FLASHOPT_PAIRS_MAX || tokens < 0 || tokens > int64_t(1) << 40)
        return FLASHOPT_ERR_SIZE;
    if (!std::isfinite(beta) || !std::isfinite(margin) || !(smoothing >= 0.0 && smoothing <= 1.0) ||
        average < 0 || average > 1)
        return FLASHOPT_ERR_ARG;
    return FLASHOPT_OK;
}

static unsigned token_grid(int64_t n) {
    const int64_t blocks = (n + kBlock - 1) / kBlock;
    return (unsigned)(blocks < 65536 ? blocks : 65536);
}

int launch_preference(const PreferenceIn& in, void* workspace, hipStream_t st) {
    if (in.pairs == 0) {
        if (!in.grad || in.tokens == 0) return FLASHOPT_OK;
        hipLaunchKernelGGL(no_pairs_kernel, dim3(token_grid(in.tokens)), dim3(kBlock), 0, st, in.grad, in.tokens);
        return launch_status();
    }
    const int shares = (int)shares_of(in.pairs, in.tokens);
    const dim3 grid((unsigned)(in.pairs * shares)), block(kPairThreads);
    PairSums* parts = (PairSums*)workspace;
    if (shares == 1) {
        hipLaunchKernelGGL((preference_kernel<0>), grid, block, 0, st, in, 1, nullptr);
    } else {
        hipLaunchKernelGGL((preference_kernel<1>), grid, block, 0, st, in, shares, parts);
        hipLaunchKernelGGL((preference_kernel<2>), grid, block, 0, st, in, shares, parts);
    }
    return launch_status();
}

}  // namespace flashopt

using namespace flashopt;

extern "C" {

int flashopt_policy(const float* logprob, const float* old_logprob, const float* advantage,
                    const float* ref_logprob, const float* weight, const uint8_t* mask, int64_t n,
                    double clip_low, double clip_high, double kl, const float* grad_loss,
                    float* loss, float* grad_logprob, void* stream) {
    if (n < 0 || n > int64_t(1) << 40) return FLASHOPT_ERR_SIZE;
    PolicyIn in;
    const int e = policy_terms(n, clip_low, clip_high, kl, 0.0, ref_logprob, in);
    if (e) return e;
    if (n == 0) return FLASHOPT_OK;
    if (!logprob || !old_logprob || !advantage) return FLASHOPT_ERR_NULL;
    if (!aligned(logprob, 4) || !aligned(old_logprob, 4) || !aligned(advantage, 4) ||
        !aligned(ref_logprob, 4) || !aligned(weight, 4) || !aligned(grad_loss, 4) || !aligned(loss, 4) ||
        !aligned(grad_logprob, 4))
        return FLASHOPT_ERR_ALIGN;
    if (!loss && !grad_logprob) return FLASHOPT_OK;
    in.old = old_logprob;
    in.advantage = advantage;
    in.weight = weight;
    in.loss = loss;
    hipLaunchKernelGGL(policy_kernel, dim3(token_grid(n)), dim3(kBlock), 0, (hipStream_t)stream, logprob,
                       in, mask, n, grad_loss, grad_logprob);
    return launch_status();
}

size_t flashopt_preference_workspace_bytes(int64_t pairs, int64_t tokens) {
    return check_preference(pairs, tokens, 0.0, 0.0, 0.0, 0) ? 0 : preference_workspace(pairs, tokens);
}

int flashopt_preference(const float* logprob, const float* ref_logprob, const uint8_t* mask,
                        int64_t tokens, const int64_t* offsets, int64_t pairs, double beta,
                        double margin, double smoothing, int32_t average, const float* grad_loss,
                        void* workspace, size_t workspace_bytes, float* loss, float* reward,
                        float* grad_logprob, void* stream) {
    const int e = check_preference(pairs, tokens, beta, margin, smoothing, average);
    if (e) return e;
    if ((pairs > 0 && !offsets) || (pairs > 0 && tokens > 0 && !logprob)) return FLASHOPT_ERR_NULL;
    if (!aligned(logprob, 4) || !aligned(ref_logprob, 4) || !aligned(offsets, 8) || !aligned(grad_loss, 4) ||
        !aligned(loss, 4) || !aligned(reward, 4) || !aligned(grad_logprob, 4))
        return FLASHOPT_ERR_ALIGN;
    const size_t need = preference_workspace(pairs, tokens);
    if (need && !workspace) return FLASHOPT_ERR_NULL;
    if (need && (workspace_bytes < need || !aligned(workspace, 256))) return FLASHOPT_ERR_WORKSPACE;
    return launch_preference({logprob, ref_logprob, mask, nullptr, 0, offsets, pairs, tokens, beta, margin,
                              smoothing, average, grad_loss, loss, reward, grad_logprob},
                             workspace, (hipStream_t)stream);
}

}  // extern "C"
