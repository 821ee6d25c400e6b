// Log-probabilities of given tokens, with entropy and the top alternatives,
// and their gradient.
#include "common.cuh"
#include "launch.h"

namespace {

constexpr int LP_NT = 256;

// A logit's place in the order (larger logits larger; -0 as 0) above its
// column's (lower columns larger): unique within a row.
__device__ __forceinline__ uint64_t order_key(float z, int col) {
    const int b = __float_as_int(z + 0.f);
    const uint32_t u = (uint32_t)(b < 0 ? ~b : b ^ 0x80000000);
    return ((uint64_t)u << 32) | (uint32_t)~col;
}

template <typename T>
__global__ void __launch_bounds__(LP_NT)
    logprobs_kernel(float* logp, float* lse, float* entropy, float* top_logp, int32_t* top_ids, int k,
                    const T* logits, const int32_t* targets, int N, int V, int Vp, int* status) {
    __shared__ float sh[3][LP_NT];
    __shared__ uint64_t best[LP_NT];
    const int row = blockIdx.x, tid = threadIdx.x;
    const T* z = logits + (int64_t)row * Vp;
    float m = -INFINITY;
    for (int j = tid; j < V; j += LP_NT) {
        const float x = to_float(z[j]);
        m = x > m || x != x ? x : m;
    }
    sh[0][tid] = m;
    __syncthreads();
    for (int w = LP_NT / 2; w > 0; w /= 2) {
        if (tid < w) {
            const float x = sh[0][tid], y = sh[0][tid + w];
            sh[0][tid] = y > x || y != y ? y : x;
        }
        __syncthreads();
    }
    m = sh[0][0];
    float s = 0.f, t = 0.f;
    for (int j = tid; j < V; j += LP_NT) {
        const float d = to_float(z[j]) - m, e = expf(d);
        s += e;
        if (!(e == 0.f)) t += e * d;
    }
    sh[1][tid] = s;
    sh[2][tid] = t;
    __syncthreads();
    for (int w = LP_NT / 2; w > 0; w /= 2) {
        if (tid < w) {
            sh[1][tid] += sh[1][tid + w];
            sh[2][tid] += sh[2][tid + w];
        }
        __syncthreads();
    }
    s = sh[1][0];
    t = sh[2][0];
    const bool none = m == -INFINITY;
    const float L = isinf(m) ? m : m + logf(s);
    if (tid == 0) {
        lse[row] = L;
        if (entropy) entropy[row] = none ? 0.f : logf(s) - t / s;
        if (logp) {
            int tgt = targets[row];
            if (tgt < 0 || tgt >= V) {
                set_status(status, GPT2_FLAG_TARGET_RANGE);
                tgt = 0;
            }
            logp[row] = none ? -INFINITY : to_float(z[tgt]) - L;
        }
    }
    uint64_t last = ~0ull;
    for (int r = 0; r < k; r++) {
        uint64_t b = 0;
        for (int j = tid; j < V; j += LP_NT) {
            const uint64_t x = order_key(to_float(z[j]), j);
            if (x < last && x > b) b = x;
        }
        best[tid] = b;
        __syncthreads();
        for (int w = LP_NT / 2; w > 0; w /= 2) {
            if (tid < w && best[tid + w] > best[tid]) best[tid] = best[tid + w];
            __syncthreads();
        }
        last = best[0];
        const int col = (int)~(uint32_t)last;
        if (tid == 0) {
            top_ids[(int64_t)row * k + r] = col;
            top_logp[(int64_t)row * k + r] = none ? -INFINITY : to_float(z[col]) - L;
        }
        __syncthreads();
    }
}

template <typename T>
__global__ void __launch_bounds__(LP_NT)
    logprobs_bwd_kernel(T* dlogits, const T* logits, const int32_t* targets, const float* lse, const float* entropy,
                        const float* dlogp, const float* dlse, const float* dentropy, int V, int Vp, int* status) {
    const int row = blockIdx.x;
    const T* z = logits + (int64_t)row * Vp;
    T* dz = dlogits + (int64_t)row * Vp;
    const float L = lse[row], H = dentropy ? entropy[row] : 0.f;
    const float g = dlogp ? dlogp[row] : 0.f, a = dlse ? dlse[row] : 0.f, b = dentropy ? dentropy[row] : 0.f;
    int tgt = -1;
    if (dlogp) {
        tgt = targets[row];
        if (tgt < 0 || tgt >= V) {
            if (threadIdx.x == 0) set_status(status, GPT2_FLAG_TARGET_RANGE);
            tgt = 0;
        }
    }
    for (int j = threadIdx.x; j < Vp; j += LP_NT) {
        float d = 0.f;
        if (j < V && L != -INFINITY) {
            const float lp = to_float(z[j]) - L, p = expf(lp);
            if (!(p == 0.f)) d = p * (a - g - b * (lp + H));
            if (j == tgt) d += g;
        }
        dz[j] = from_float<T>(d);
    }
}

}  // namespace

int launch_token_logprobs(int dtype, float* logp, float* lse, float* entropy, float* top_logp, int32_t* top_ids,
                          int k, const void* logits, const int32_t* targets, int N, int V, int Vp, int* status,
                          cudaStream_t s) {
    if (dtype == GPT2_MODE_BF16)
        logprobs_kernel<bf16><<<N, LP_NT, 0, s>>>(logp, lse, entropy, top_logp, top_ids, k, (const bf16*)logits,
                                                  targets, N, V, Vp, status);
    else
        logprobs_kernel<float><<<N, LP_NT, 0, s>>>(logp, lse, entropy, top_logp, top_ids, k, (const float*)logits,
                                                   targets, N, V, Vp, status);
    return 1;
}

int launch_token_logprobs_backward(int dtype, void* dlogits, const void* logits, const int32_t* targets,
                                   const float* lse, const float* entropy, const float* dlogp, const float* dlse,
                                   const float* dentropy, int N, int V, int Vp, int* status, cudaStream_t s) {
    if (dtype == GPT2_MODE_BF16)
        logprobs_bwd_kernel<bf16><<<N, LP_NT, 0, s>>>((bf16*)dlogits, (const bf16*)logits, targets, lse, entropy,
                                                      dlogp, dlse, dentropy, V, Vp, status);
    else
        logprobs_bwd_kernel<float><<<N, LP_NT, 0, s>>>((float*)dlogits, (const float*)logits, targets, lse, entropy,
                                                       dlogp, dlse, dentropy, V, Vp, status);
    return 1;
}
