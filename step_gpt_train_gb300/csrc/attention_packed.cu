// Causal attention over packed sequences with grouped heads: the fp32 path
// and the launchers.
#include "attention_packed.cuh"

#include <cfloat>

namespace {

template <typename T, int HD> __device__ __forceinline__ void load_row(float (&x)[HD], const T* p) {
#pragma unroll
    for (int d = 0; d < HD; d += 8) {
        float t[8];
        load8(p + d, t);
#pragma unroll
        for (int e = 0; e < 8; e++) x[d + e] = t[e];
    }
}
template <typename T, int HD> __device__ __forceinline__ void store_row(T* p, const float (&x)[HD], float s) {
#pragma unroll
    for (int d = 0; d < HD; d += 8) {
        float t[8];
#pragma unroll
        for (int e = 0; e < 8; e++) t[e] = x[d + e] * s;
        store8(p + d, t);
    }
}

// One thread per (head, query).
template <typename T, int HD> __global__ void __launch_bounds__(128) packed_fwd_kernel(PackedAttn a, float scale) {
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
    float q[HD], acc[HD];
    load_row<T, HD>(q, (const T*)a.q + row * a.q_stride + h * HD);
#pragma unroll
    for (int d = 0; d < HD; d++) acc[d] = 0.f;
    float m = -INFINITY, l = 0.f;
    const int n = min(t + p.lk - p.lq + 1, p.lk);
    for (int j = 0; j < n; j++) {
        float x[HD];
        load_row<T, HD>(x, (const T*)a.k + (p.k0 + j) * a.k_stride + hk * HD);
        float sc = 0.f;
#pragma unroll
        for (int d = 0; d < HD; d++) sc += q[d] * x[d];
        sc *= scale;
        if (sc > m) {
            const float f = m == -INFINITY ? 0.f : expf(m - sc);
            l *= f;
#pragma unroll
            for (int d = 0; d < HD; d++) acc[d] *= f;
            m = sc;
        }
        const float w = m == -INFINITY ? (sc == sc ? 0.f : sc) : expf(sc - m);
        l += w;
        load_row<T, HD>(x, (const T*)a.v + (p.k0 + j) * a.v_stride + hk * HD);
#pragma unroll
        for (int d = 0; d < HD; d++) acc[d] += w * x[d];
    }
    store_row<T, HD>((T*)a.o + row * a.o_stride + h * HD, acc, l == 0.f ? 0.f : 1.f / l);
    a.lse[(int64_t)h * a.total_q + row] = l == 0.f ? -INFINITY : m + logf(l);
}

// One thread per (head, query): dQ, and D for the other kernel.
template <typename T, int HD>
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
    load_row<T, HD>(q, (const T*)a.o + row * a.o_stride + h * HD);
    load_row<T, HD>(dy, (const T*)g.dout + row * g.dout_stride + h * HD);
#pragma unroll
    for (int d = 0; d < HD; d++) D += q[d] * dy[d];
    g.D[(int64_t)h * a.total_q + row] = D;
    load_row<T, HD>(q, (const T*)a.q + row * a.q_stride + h * HD);
#pragma unroll
    for (int d = 0; d < HD; d++) dq[d] = 0.f;
    const float L = a.lse[(int64_t)h * a.total_q + row];
    const int n = min(t + p.lk - p.lq + 1, p.lk);
    for (int j = 0; j < n; j++) {
        float k[HD], v[HD];
        load_row<T, HD>(k, (const T*)a.k + (p.k0 + j) * a.k_stride + hk * HD);
        load_row<T, HD>(v, (const T*)a.v + (p.k0 + j) * a.v_stride + hk * HD);
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
    store_row<T, HD>((T*)g.dq + row * g.dq_stride + h * HD, dq, scale);
}

// One thread per (key head, key).
template <typename T, int HD>
__global__ void __launch_bounds__(128) packed_dkdv_kernel(PackedAttn a, PackedAttnGrad g, float scale) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= a.total_k * a.Hkv) return;
    const int hk = i / a.total_k, row = i - hk * a.total_k;
    const int s = packed_find_row(a.cu_k, a.n_seq, row);
    if (s < 0) return;
    const PackedSeq p = packed_seq(a, s);
    const int j = row - p.k0;
    if (j < 0 || j >= p.lk) return;
    const int group = a.Hq / a.Hkv;
    float k[HD], v[HD], dk[HD], dv[HD];
    load_row<T, HD>(k, (const T*)a.k + row * a.k_stride + hk * HD);
    load_row<T, HD>(v, (const T*)a.v + row * a.v_stride + hk * HD);
#pragma unroll
    for (int d = 0; d < HD; d++) dk[d] = dv[d] = 0.f;
    for (int h = hk * group; h < (hk + 1) * group; h++)
        for (int t = max(0, j - (p.lk - p.lq)); t < p.lq; t++) {
            float q[HD], dy[HD];
            const int64_t r = p.q0 + t;
            load_row<T, HD>(q, (const T*)a.q + r * a.q_stride + h * HD);
            load_row<T, HD>(dy, (const T*)g.dout + r * g.dout_stride + h * HD);
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
    store_row<T, HD>((T*)g.dk + row * g.dk_stride + hk * HD, dk, scale);
    store_row<T, HD>((T*)g.dv + row * g.dv_stride + hk * HD, dv, 1.f);
}

// The tiles of a call sorted by their key blocks, most first (a counting sort
// in one block; equal ones in any order, which changes no result), and the
// counter set to 0. Longest first from one counter leaves the SMs within a
// short item of each other at the end: dealt round robin in sequence order
// they were busy two thirds of the time on 16 ragged prompts.
constexpr int PLAN_SEQ = 2048;  // sequences whose offsets are searched in shared memory
struct PlanArgs {
    PackedCut cut[2];
    PackedPlan* plan[2];
};
__global__ void __launch_bounds__(1024) packed_plan_kernel(PackedAttn a, PlanArgs args) {
    const PackedCut cut = args.cut[blockIdx.x];
    PackedPlan* plan = args.plan[blockIdx.x];
    const int slots = cut.slots(a), per = cut.per, total = cut.total(a);
    constexpr int BUCKETS = 1024;
    __shared__ int count[BUCKETS], warps[32], first[PLAN_SEQ], keys[PLAN_SEQ + 1], rows[PLAN_SEQ + 1];
    const int tid = threadIdx.x, lane = tid & 31;
    const bool near = a.n_seq <= PLAN_SEQ;
    if (near)
        for (int s = tid; s <= a.n_seq; s += 1024) {
            rows[s] = a.cu_q[s];
            keys[s] = a.cu_k[s];
            if (s < a.n_seq) first[s] = min(max((cut.keys ? keys : rows)[s], 0), total) / per + s;
        }
    count[tid] = 0;
    __syncthreads();
    PackedAttn c = a;
    if (near) c.cu_q = rows, c.cu_k = keys;
    if (blockIdx.x == 0) packed_check(c, tid, 1024);
    // the tile of a slot, its bucket, or -1
    auto look = [&](int slot, PackedTile& t) -> int {
        int lo = -1, hi = a.n_seq, f = 0;  // the last sequence whose first slot is at or before this one
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            const int x = near ? first[mid] : min(max(cut.cu(a)[mid], 0), total) / per + mid;
            if (x <= slot) lo = mid, f = x;
            else hi = mid;
        }
        if (lo < 0) return -1;
        const PackedSeq p = packed_seq(c, lo);
        const int at = (slot - f) * per;
        if (at < 0 || at >= cut.rows(p)) return -1;
        t = cut.tile(p, at);
        return BUCKETS - 1 - min(cut.blocks(t, t.n), BUCKETS - 1);
    };
    PackedTile t0;
    const int b0 = tid < slots ? look(tid, t0) : -1;
    if (b0 >= 0) atomicAdd(&count[b0], 1);
    for (int slot = tid + 1024; slot < slots; slot += 1024) {
        PackedTile t;
        const int b = look(slot, t);
        if (b >= 0) atomicAdd(&count[b], 1);
    }
    __syncthreads();
    {  // exclusive prefix sums over the buckets
        const int n = count[tid];
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warps[tid >> 5] = x;
        __syncthreads();
        if (tid < 32) {
            int y = warps[tid];
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int z = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) y += z;
            }
            warps[tid] = y;
        }
        __syncthreads();
        x += tid >= 32 ? warps[(tid >> 5) - 1] : 0;
        count[tid] = x - n;
        if (tid == 1023) {
            plan->count = x;
            plan->next = 0;
        }
        __syncthreads();
    }
    if (b0 >= 0) plan->tile[atomicAdd(&count[b0], 1)] = t0;
    for (int slot = tid + 1024; slot < slots; slot += 1024) {
        PackedTile t;
        const int b = look(slot, t);
        if (b >= 0) plan->tile[atomicAdd(&count[b], 1)] = t;
    }
}

template <typename T, int HD> int forward(const PackedAttn& a, cudaStream_t s) {
    packed_fwd_kernel<T, HD><<<(a.total_q * a.Hq + 127) / 128, 128, 0, s>>>(a, 1.f / sqrtf((float)HD));
    return 1;
}
template <typename T, int HD> int backward(const PackedAttn& a, const PackedAttnGrad& g, cudaStream_t s) {
    const float scale = 1.f / sqrtf((float)HD);
    if (a.total_q) packed_dq_kernel<T, HD><<<(a.total_q * a.Hq + 127) / 128, 128, 0, s>>>(a, g, scale);
    if (a.total_k) packed_dkdv_kernel<T, HD><<<(a.total_k * a.Hkv + 127) / 128, 128, 0, s>>>(a, g, scale);
    return (a.total_q > 0) + (a.total_k > 0);
}

}  // namespace

int launch_packed_plans(const PackedAttn& a, const PackedCut* cuts, PackedPlan* const* plans, int n, cudaStream_t s) {
    PlanArgs args;
    for (int i = 0; i < 2; i++) {
        args.cut[i] = cuts[i < n ? i : 0];
        args.plan[i] = plans[i < n ? i : 0];
    }
    packed_plan_kernel<<<n, 1024, 0, s>>>(a, args);
    return 1;
}

size_t attention_packed_forward_scratch(int dtype, int n_seq, int total_q, int total_k, int max_q, int max_k, int Hq,
                                        int Hkv, int hd) {
    if (dtype != GPT2_MODE_BF16) return 0;
    if (attention_packed_few(max_q, Hq, Hkv)) 
        return attention_packed_few_scratch(n_seq, total_k, max_q, max_k, Hq, Hkv);
    return attention_packed_forward_tc_scratch(n_seq, total_q, Hq, Hkv);
}

int launch_attention_packed_forward(int dtype, const PackedAttn& a, void* scratch, cudaStream_t s) {
    if (dtype == GPT2_MODE_BF16 && attention_packed_few(a.max_q, a.Hq, a.Hkv))
        return launch_attention_packed_few(a, scratch, s);
    if (dtype == GPT2_MODE_BF16) return launch_attention_packed_forward_tc(a, (PackedPlan*)scratch, s);
    return launch_attention_packed_forward_f32(a, s);
}

size_t attention_packed_backward_scratch(int dtype, int n_seq, int total_q, int total_k, int Hq, int Hkv, int hd) {
    if (dtype == GPT2_MODE_BF16 && Hq / Hkv <= 64)
        return attention_packed_backward_tc_scratch(n_seq, total_q, total_k, Hq, Hkv);
    return (size_t)Hq * total_q * 4;
}

int launch_attention_packed_backward(int dtype, const PackedAttn& a, const PackedAttnGrad& grad, void* scratch,
                                     cudaStream_t s) {
    PackedAttnGrad g = grad;
    g.D = (float*)scratch;
    if (dtype == GPT2_MODE_BF16) {
        // the tensor-core kernels lay a key head's whole group into 64 rows
        if (a.Hq / a.Hkv <= 64) return launch_attention_packed_backward_tc(a, g, scratch, s);
        return backward<bf16, 64>(a, g, s);
    }
    return launch_attention_packed_backward_f32(a, g, s);
}
