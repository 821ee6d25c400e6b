// Causal attention over packed sequences with grouped heads: the launchers, and
// the bf16 backward of groups wider than the tensor-core kernels' 64 rows (a
// thread per query or key row; MQA with 65 to 128 heads). It is the simple form,
// bound by each thread's chain of loads: 4 sequences of 300 tokens and 128 heads
// on one take 63 ms (64 heads on the tensor cores: 0.23).
#include "attention_packed.cuh"

namespace {

constexpr int HD = 64;

__device__ __forceinline__ void load_row(float (&x)[HD], const bf16* p) {
#pragma unroll
    for (int d = 0; d < HD; d += 8) {
        float t[8];
        load8(p + d, t);
#pragma unroll
        for (int e = 0; e < 8; e++) x[d + e] = t[e];
    }
}
__device__ __forceinline__ void store_row(bf16* p, const float (&x)[HD], float s) {
#pragma unroll
    for (int d = 0; d < HD; d += 8) {
        float t[8];
#pragma unroll
        for (int e = 0; e < 8; e++) t[e] = x[d + e] * s;
        store8(p + d, t);
    }
}

// One thread per (head, query): dQ, and D for the other kernel.
__global__ void __launch_bounds__(128) packed_dq_kernel(PackedAttn a, PackedAttnGrad g, float scale) {
    const int i = blockIdx.x * 128 + threadIdx.x;  // both counts stay below 2^30
    packed_check(a, i, gridDim.x * 128);
    if (i >= a.total_q * a.Hq) return;
    const int h = i / a.total_q, row = i - h * a.total_q;
    const int s = packed_find_row(a.cu_q, a.n_seq, row);
    if (s < 0) return;
    const PackedSeq p = packed_seq(a, s);
    const int t = row - p.q0;
    if (t < 0 || t >= p.lq) return;
    const int hk = h / (a.Hq / a.Hkv);
    float q[HD], dy[HD], dq[HD];
    float D = 0.f;
    load_row(q, (const bf16*)a.o + row * a.o_stride + h * HD);
    load_row(dy, (const bf16*)g.dout + row * g.dout_stride + h * HD);
#pragma unroll
    for (int d = 0; d < HD; d++) D += q[d] * dy[d];
    g.D[(int64_t)h * a.total_q + row] = D;
    load_row(q, (const bf16*)a.q + row * a.q_stride + h * HD);
#pragma unroll
    for (int d = 0; d < HD; d++) dq[d] = 0.f;
    const float L = a.lse[(int64_t)h * a.total_q + row];
    const int n = min(t + p.lk - p.lq + 1, p.lk);
    for (int j = 0; j < n; j++) {
        float k[HD], v[HD];
        load_row(k, (const bf16*)a.k + (p.k0 + j) * a.k_stride + hk * HD);
        load_row(v, (const bf16*)a.v + (p.k0 + j) * a.v_stride + hk * HD);
        float sc = 0.f, dp = 0.f;
#pragma unroll
        for (int d = 0; d < HD; d++) {
            sc += q[d] * k[d];
            dp += dy[d] * v[d];
        }
        const float ds = expf(sc * scale - L) * (dp - D);
#pragma unroll
        for (int d = 0; d < HD; d++) dq[d] += ds * k[d];
    }
    store_row((bf16*)g.dq + row * g.dq_stride + h * HD, dq, scale);
}

// One thread per (key head, key).
__global__ void __launch_bounds__(128) packed_dkdv_kernel(PackedAttn a, PackedAttnGrad g, float scale) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (a.total_q == 0) packed_check(a, i, gridDim.x * blockDim.x);  // (else the other kernel looks)
    if (i >= a.total_k * a.Hkv) return;
    const int hk = i / a.total_k, row = i - hk * a.total_k;
    const int s = packed_find_row(a.cu_k, a.n_seq, row);
    if (s < 0) return;
    const PackedSeq p = packed_seq(a, s);
    const int j = row - p.k0;
    if (j < 0 || j >= p.lk) return;
    const int group = a.Hq / a.Hkv;
    float k[HD], v[HD], dk[HD], dv[HD];
    load_row(k, (const bf16*)a.k + row * a.k_stride + hk * HD);
    load_row(v, (const bf16*)a.v + row * a.v_stride + hk * HD);
#pragma unroll
    for (int d = 0; d < HD; d++) dk[d] = dv[d] = 0.f;
    for (int h = hk * group; h < (hk + 1) * group; h++)
        for (int t = max(0, j - (p.lk - p.lq)); t < p.lq; t++) {
            float q[HD], dy[HD];
            const int64_t r = p.q0 + t;
            load_row(q, (const bf16*)a.q + r * a.q_stride + h * HD);
            load_row(dy, (const bf16*)g.dout + r * g.dout_stride + h * HD);
            float sc = 0.f, dp = 0.f;
#pragma unroll
            for (int d = 0; d < HD; d++) {
                sc += q[d] * k[d];
                dp += dy[d] * v[d];
            }
            const float w = expf(sc * scale - a.lse[h * (int64_t)a.total_q + r]);
            const float ds = w * (dp - g.D[h * (int64_t)a.total_q + r]);
#pragma unroll
            for (int d = 0; d < HD; d++) {
                dv[d] += w * dy[d];
                dk[d] += ds * q[d];
            }
        }
    store_row((bf16*)g.dk + row * g.dk_stride + hk * HD, dk, scale);
    store_row((bf16*)g.dv + row * g.dv_stride + hk * HD, dv, 1.f);
}

int backward_wide(const PackedAttn& a, const PackedAttnGrad& g, cudaStream_t s) {
    const float scale = 1.f / sqrtf((float)HD);
    if (a.total_q) packed_dq_kernel<<<(a.total_q * a.Hq + 127) / 128, 128, 0, s>>>(a, g, scale);
    if (a.total_k) packed_dkdv_kernel<<<(a.total_k * a.Hkv + 127) / 128, 128, 0, s>>>(a, g, scale);
    return (a.total_q > 0) + (a.total_k > 0);
}

}  // namespace

size_t attention_packed_forward_scratch(int dtype, int n_seq, int total_q, int total_k, int max_q, int max_k, int Hq,
                                        int Hkv, int hd) {
    if (dtype != GPT2_MODE_BF16) return attention_packed_forward_f32_scratch(n_seq, total_q, Hq, Hkv);
    if (attention_packed_few(max_q, Hq, Hkv))
        return attention_packed_few_scratch(n_seq, total_k, max_q, max_k, Hq, Hkv);
    return attention_packed_forward_tc_scratch(n_seq, total_q, Hq, Hkv);
}

int launch_attention_packed_forward(int dtype, const PackedAttn& a, void* scratch, cudaStream_t s) {
    if (dtype == GPT2_MODE_BF16 && attention_packed_few(a.max_q, a.Hq, a.Hkv))
        return launch_attention_packed_few(a, scratch, s);
    if (dtype == GPT2_MODE_BF16) return launch_attention_packed_forward_tc(a, (PackedPlan*)scratch, s);
    return launch_attention_packed_forward_f32(a, (PackedPlan*)scratch, s);
}

size_t attention_packed_backward_scratch(int dtype, int n_seq, int total_q, int total_k, int Hq, int Hkv, int hd) {
    if (dtype != GPT2_MODE_BF16) return 0;
    if (Hq / Hkv <= 64) return attention_packed_backward_tc_scratch(n_seq, total_q, total_k, Hq, Hkv);
    return (size_t)Hq * total_q * 4;  // D
}

int launch_attention_packed_backward(int dtype, const PackedAttn& a, const PackedAttnGrad& grad, void* scratch,
                                     cudaStream_t s) {
    PackedAttnGrad g = grad;
    g.D = (float*)scratch;
    if (dtype == GPT2_MODE_BF16) {
        // the tensor-core kernels lay a key head's whole group into 64 rows
        if (a.Hq / a.Hkv <= 64) return launch_attention_packed_backward_tc(a, g, scratch, s);
        return backward_wide(a, g, s);
    }
    return launch_attention_packed_backward_f32(a, g, s);
}
