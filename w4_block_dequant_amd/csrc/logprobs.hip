// Log probabilities of given tokens, entropy and the largest entries, read off
// the head's logits (see include/w4.h).  With m = max x, S = sum e^(x-m):
//   log p = (x - m) - log S,   entropy = log S - (sum e^(x-m) (x-m)) / S.
//
// One workgroup takes one row: its maximum, then the two sums, then one pass
// for each of the largest entries (the largest key below the last one; a key
// holds the value and the inverted index, so ties go to the lower index).
#include <math.h>

#include "kv.h"
#include "launch.h"

namespace w4 {
namespace {

constexpr int kThreads = 256;

template <class T, class F>
__device__ __forceinline__ T block_reduce(T v, T *s, F f) {
    __syncthreads();
    s[threadIdx.x] = v;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        if (threadIdx.x < (unsigned)o) s[threadIdx.x] = f(s[threadIdx.x], s[threadIdx.x + o]);
        __syncthreads();
    }
    return s[0];
}

__global__ __launch_bounds__(kThreads) void k_logprobs(const float *logits, int64_t N, int64_t ld,
                                                       const int64_t *tokens, int top,
                                                       float *logprob, float *entropy,
                                                       int64_t *top_ids, float *top_logprob,
                                                       int *d_status) {
    __shared__ float sf[kThreads];
    __shared__ uint64_t su[kThreads];
    const int64_t row = blockIdx.x;
    const float *x = logits + row * ld;
    float m = -INFINITY;
    int bad = 0;
    for (int64_t n = threadIdx.x; n < N; n += kThreads) {
        bad |= !(x[n] < INFINITY);
        m = fmaxf(m, x[n]);
    }
    m = block_reduce(m, sf, [](float a, float b) { return fmaxf(a, b); });
    bad = block_reduce((float)bad, sf, [](float a, float b) { return a + b; }) != 0.0f;
    const bool none = m == -INFINITY && !bad;
    float S = 0.0f, W = 0.0f;
    for (int64_t n = threadIdx.x; n < N; n += kThreads) {
        const float d = x[n] - m;  // -infinity where the difference passes fp32
        const float e = expf(d);
        if (e > 0.0f) {
            S += e;
            W += e * d;
        }
    }
    auto add = [](float a, float b) { return a + b; };
    S = block_reduce(S, sf, add);
    W = block_reduce(W, sf, add);
    const float logS = logf(S);
    auto log_p = [&](float v) {
        return bad ? NAN : none || v == -INFINITY ? -INFINITY : (v - m) - logS;
    };
    if (threadIdx.x == 0) {
        if (bad) set_status(d_status, W4_ERR_NONFINITE);
        if (logprob) {
            const int64_t token = tokens[row];
            const bool in = token >= 0 && token < N;
            if (!in) set_status(d_status, W4_ERR_BAD_SHAPE);
            logprob[row] = in ? log_p(x[token]) : NAN;
        }
        if (entropy) entropy[row] = bad ? NAN : none ? 0.0f : logS - W / S;
    }
    uint64_t last = ~0ull;
    for (int j = 0; j < top; ++j) {
        uint64_t best = 0;
        for (int64_t n = threadIdx.x; n < N; n += kThreads) {
            const uint64_t key = (uint64_t)order_key(x[n]) << 32 | (uint32_t)~(uint32_t)n;
            if (key < last && key > best) best = key;
        }
        best = block_reduce(best, su, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
        last = best;
        if (threadIdx.x == 0) {
            top_ids[row * top + j] = bad ? -1 : (int64_t)(uint32_t)~(uint32_t)best;
            top_logprob[row * top + j] = log_p(order_value((uint32_t)(best >> 32)));
        }
    }
}

}  // namespace

size_t logprobs_workspace(int64_t M, int64_t N, int64_t top) {
    (void)M, (void)N, (void)top;
    return 0;
}

hipError_t launch_logprobs(const float *logits, int64_t M, int64_t N, int64_t ld,
                           const int64_t *tokens, int64_t top, float *logprob, float *entropy,
                           int64_t *top_ids, float *top_logprob, void *workspace, int *d_status,
                           hipStream_t stream) {
    (void)workspace;
    hipLaunchKernelGGL(k_logprobs, dim3((unsigned)M), dim3(kThreads), 0, stream, logits, N, ld,
                       tokens, (int)top, logprob, entropy, top_ids, top_logprob, d_status);
    return hipGetLastError();
}

}  // namespace w4
