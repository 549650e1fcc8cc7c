// lb_token_logprobs: per row x of logits, with m = max x and S = sum e^(x - m),
//   log p_i = (x_i - m) - log S,
//   entropy = -sum p_i log p_i = log S - sum e^(x - m) (x - m) / S,
// the log probabilities of the given tokens and of the `top` largest logits.
// Both terms of the entropy are >= 0, so nothing cancels.
#include <cmath>

#include "lb_dense.cuh"

namespace lb {
namespace {

constexpr int kLpThreads = 256;
constexpr int kMaxTop = 32;

struct LogprobArgs {
    const void* x;
    const int64_t* tokens;
    float* logprob;
    float* entropy;
    int64_t* top_id;
    float* top_logprob;
    int64_t ld;
    int vocab, top;
};

// Order of the alternatives as an unsigned key: larger logit first, NaN before
// everything, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 0xffffffffu;
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One block per row; `top` rounds, each the largest (key, lowest index) below
// the one before it.
template <int DT>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const LogprobArgs a) {
    using X = Elem<DT>;
    __shared__ float fred[3][kLpThreads / 32];
    __shared__ unsigned long long kred[kLpThreads / 32];
    const int64_t row = blockIdx.x;
    const typename X::T* x = static_cast<const typename X::T*>(a.x) + row * a.ld;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float m = -INFINITY;
    bool nan = false;
    for (int i = threadIdx.x; i < a.vocab; i += kLpThreads) {
        const float v = X::get(x[i]);
        nan |= v != v;
        m = fmaxf(m, v);
    }
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) fred[0][warp] = m;
    nan = __syncthreads_or(nan) != 0;
    for (int w = 0; w < kLpThreads / 32; ++w) m = fmaxf(m, fred[0][w]);
    const bool empty = m == -INFINITY && !nan;
    float S = 0.0f, A = 0.0f;
    if (!empty)
        for (int i = threadIdx.x; i < a.vocab; i += kLpThreads) {
            const float d = X::get(x[i]) - m, e = expf(d);
            S += e;
            if (e > 0.0f) A += e * d;
        }
    for (int o = 16; o > 0; o >>= 1) {
        S += __shfl_xor_sync(0xffffffffu, S, o);
        A += __shfl_xor_sync(0xffffffffu, A, o);
    }
    if (lane == 0) { fred[1][warp] = S; fred[2][warp] = A; }
    __syncthreads();
    S = A = 0.0f;
    for (int w = 0; w < kLpThreads / 32; ++w) { S += fred[1][w]; A += fred[2][w]; }
    const bool bad = nan || m == INFINITY;
    const float logS = logf(S);
    auto logprob = [&](float v) { return bad ? NAN : empty ? -INFINITY : (v - m) - logS; };
    if (threadIdx.x == 0) {
        if (a.entropy) a.entropy[row] = bad ? NAN : empty ? 0.0f : logS - A / S;
        if (a.tokens) {
            const int64_t t = a.tokens[row];
            a.logprob[row] = t < 0 ? 0.0f : t >= a.vocab ? NAN : logprob(X::get(x[t]));
        }
    }
    unsigned long long last = ~0ull;
    for (int k = 0; k < a.top; ++k) {
        unsigned long long best = 0;
        for (int i = threadIdx.x; i < a.vocab; i += kLpThreads) {
            const unsigned long long c = (unsigned long long)order_key(X::get(x[i])) << 32 | (0xffffffffu - i);
            if (c < last && c > best) best = c;
        }
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long c = __shfl_xor_sync(0xffffffffu, best, o);
            best = c > best ? c : best;
        }
        __syncthreads();
        if (lane == 0) kred[warp] = best;
        __syncthreads();
        for (int w = 0; w < kLpThreads / 32; ++w) best = kred[w] > best ? kred[w] : best;
        last = best;
        if (threadIdx.x == 0) {
            const int i = (int)(0xffffffffu - (uint32_t)best);
            a.top_id[row * a.top + k] = i;
            a.top_logprob[row * a.top + k] = logprob(X::get(x[i]));
        }
    }
}

}  // namespace
}  // namespace lb

using namespace lb;

extern "C" lb_status lb_token_logprobs(const void* logits, lb_dtype dtype, int64_t rows,
                                       int64_t vocab, int64_t ld, const int64_t* tokens,
                                       float* logprob, float* entropy, int top, int64_t* top_id,
                                       float* top_logprob, void* stream) {
    if (!logits || !dtype_ok(dtype)) return LB_ERR_INVALID_ARG;
    if (rows <= 0 || rows > 0x7fffffff || vocab <= 0 || vocab > (1 << 24) || ld < vocab ||
        ld > ((int64_t)1 << 40))
        return LB_ERR_INVALID_ARG;
    if ((tokens != nullptr) != (logprob != nullptr)) return LB_ERR_INVALID_ARG;
    if (top < 0 || top > kMaxTop || top > vocab) return LB_ERR_INVALID_ARG;
    if (top > 0 && (!top_id || !top_logprob)) return LB_ERR_INVALID_ARG;
    if (!tokens && !entropy && top == 0) return LB_ERR_INVALID_ARG;
    if (!is_aligned(logits, dtype_size(dtype)) || !is_aligned(tokens, 8) || !is_aligned(logprob, 4) ||
        !is_aligned(entropy, 4) || (top > 0 && (!is_aligned(top_id, 8) || !is_aligned(top_logprob, 4))))
        return LB_ERR_ALIGNMENT;
    const lb_status st = dense_device_ok();
    if (st != LB_OK) return st;
    const LogprobArgs a = {logits, tokens, logprob, entropy, top_id, top_logprob, ld, (int)vocab, top};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    with_dtype(dtype, [&](auto d) { logprobs_kernel<d.value><<<(unsigned)rows, kLpThreads, 0, s>>>(a); });
    return cudaGetLastError() == cudaSuccess ? LB_OK : LB_ERR_CUDA;
}
