// Softmax cross entropy over a large vocabulary from hidden states and the
// head's weight, without keeping the logits (gpt2_op_linear_classifier_*).
//
//   z = x W^T, lse = ln sum_j<V exp z_j, loss = lse - z_target
//   dz = (dloss + dlse) exp(z - lse) - dloss [j = target], dx = dz W, dW = dz^T x
//
// bf16: the forward is one tensor-core matmul whose epilogue reduces each row
// of a half tile to its maximum and sum of exponentials (gemm_tc.cu, EPI_LSE);
// a second kernel joins a row's parts. The logits are never rounded to bf16.
// The backward goes through the vocabulary in pieces: the same matmul with an
// epilogue that writes the piece of dz in bf16 (EPI_DZ), then both products
// that read it. Pieces of the vocabulary, not of the rows: a piece's rows of
// dW are whole, and what is added to from piece to piece is dx, N x C values,
// where pieces of rows would add to V x C. Its values are added in fp32 by the
// copies that store them (one writer for each value in a launch, so the order
// is fixed).
//
// fp32: the same with the fp32 matmul and the logits of a piece in scratch.
#include "common.cuh"
#include "launch.h"

namespace {

constexpr float LOG2E = 1.4426950408889634f;

// What one piece of dz may take; see pieces().
constexpr int64_t PIECE_BYTES = 256ll << 20;

struct Pieces {
    int width, n;
};
// Pieces of equal width, in steps of a tile, that hold PIECE_BYTES for all rows (but no fewer than 2048 columns).
Pieces pieces(int dtype, int N, int V) {
    const int64_t es = dtype == GPT2_MODE_BF16 ? 2 : 4;
    int64_t most = PIECE_BYTES / ((int64_t)N * es);
    if (most < 2048) most = 2048;
    const int n = (int)((V + most - 1) / most);
    const int width = ((V + n - 1) / n + 255) / 256 * 256;
    return {width, (V + width - 1) / width};
}
int round8(int v) { return (v + 7) / 8 * 8; }
size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Joins the parts of 32 rows: strand after strand of slots (a warp's lanes read neighbouring rows of one slot),
// then the strands. Loads run ahead in batches: a part's exponentials wait for it, the next parts do not.
// 8 strands where there are rows enough to fill the device with them, 32 for fewer rows.
template <int STRANDS, int AHEAD>
__global__ void __launch_bounds__(STRANDS * 32) join_kernel(float* __restrict__ losses, float* __restrict__ lse,
                                                           const float2* __restrict__ stats,
                                                           const float* __restrict__ target_logit,
                                                           const int32_t* __restrict__ targets, int N, int V, int slots,
                                                           int* status) {
    __shared__ float2 sm[STRANDS][32];
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const int64_t row = (int64_t)blockIdx.x * 32 + tx;
    float m = -INFINITY, s = 0.f;
    auto join = [&](float2 p) {
        if (p.y == 0.f) return;  // a part without columns
        const float mm = fmaxf(m, p.x);
        s = s * ex2_approx((m - mm) * LOG2E) + p.y * ex2_approx((p.x - mm) * LOG2E);
        m = mm;
    };
    for (int i = ty; i < slots; i += STRANDS * AHEAD) {
        float2 p[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; u++) {
            const int slot = i + u * STRANDS;
            p[u] = slot < slots && row < N ? __ldcs(&stats[(int64_t)slot * N + row]) : make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < AHEAD; u++) join(p[u]);
    }
    sm[ty][tx] = make_float2(m, s);
    for (int w = STRANDS / 2; w > 0; w /= 2) {  // halves of the strands, in a fixed order
        __syncthreads();
        if (ty < w) {
            join(sm[ty + w][tx]);
            sm[ty][tx] = make_float2(m, s);
        }
    }
    if (ty || row >= N) return;
    const int t = targets[row];
    if (t < 0 || t >= V) set_status(status, GPT2_FLAG_TARGET_RANGE);
    // (max - z) + ln S rather than lse - z: a sure token's loss keeps its digits wherever the logits lie, and
    // none is negative
    const float ls = logf(s), loss = (m - target_logit[row]) + ls;
    lse[row] = m + ls;
    losses[row] = loss < 0.f ? 0.f : loss;
}

// fp32: a row's maximum and sum over a piece of the logits, and its target's logit. One warp a row.
__global__ void __launch_bounds__(256) piece_stats_kernel(float2* __restrict__ stats, float* __restrict__ target_logit,
                                                          const float* __restrict__ z,
                                                          const int32_t* __restrict__ targets, int N, int cols,
                                                          int first, int V) {
    const int lane = threadIdx.x % 32;
    const int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    if (row >= N) return;
    const float* p = z + row * cols;
    float m = -INFINITY;
    for (int i = lane; i < cols; i += 32) m = fmaxf(m, p[i]);
    m = warp_max(m);
    float s = 0.f;
    for (int i = lane; i < cols; i += 32) s += expf(p[i] - m);
    s = warp_sum(s);
    if (lane) return;
    stats[row] = make_float2(m, s);
    int t = targets[row];
    if (t < 0 || t >= V) t = 0;
    if (t >= first && t < first + cols) target_logit[row] = p[t - first];
}

// fp32: a piece of the logits becomes its gradient.
__global__ void __launch_bounds__(256) piece_dz_kernel(float* __restrict__ z, const int32_t* __restrict__ targets,
                                                       const float* __restrict__ lse, const float* __restrict__ dloss,
                                                       const float* __restrict__ dlse, int N, int cols, int first,
                                                       int V) {
    const int64_t row = blockIdx.y;
    int t = targets[row];
    if (t < 0 || t >= V) t = 0;
    const float d = dloss ? dloss[row] : 0.f, a = d + (dlse ? dlse[row] : 0.f), l = lse[row];
    for (int j = blockIdx.x * 256 + threadIdx.x; j < cols; j += gridDim.x * 256) {
        float* p = z + row * cols + j;
        const float e = a != 0.f || d != 0.f ? a * expf(*p - l) : 0.f;
        *p = e - (first + j == t ? d : 0.f);
    }
}

__global__ void __launch_bounds__(256) round_kernel(bf16* __restrict__ out, const float* __restrict__ in, int64_t n) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= n) return;
    float f[8];
    load8(in + i, f);
    store8(out + i, f);
}

// Targets out of range, in the backward.
__global__ void __launch_bounds__(256) check_targets_kernel(const int32_t* __restrict__ targets, int N, int V,
                                                            int* status) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < N && (targets[i] < 0 || targets[i] >= V)) set_status(status, GPT2_FLAG_TARGET_RANGE);
}

}  // namespace

// stats, target logits, fp32: a piece of the logits.
size_t linear_classifier_forward_scratch(int dtype, int N, int C, int V) {
    const bool bf = dtype == GPT2_MODE_BF16;
    const Pieces p = pieces(dtype, N, V);
    const int slots = bf ? head_lse_slots(N, V, C) : p.n;
    return round256((size_t)slots * N * 8) + round256((size_t)N * 4) + (bf ? 0 : (size_t)N * p.width * 4);
}

int launch_linear_classifier_forward(int dtype, float* losses, float* lse, const void* x, const void* w,
                                     const int32_t* targets, int N, int C, int V, void* scratch, int* status,
                                     cudaStream_t s) {
    const bool bf = dtype == GPT2_MODE_BF16;
    const Pieces p = pieces(dtype, N, V);
    const int slots = bf ? head_lse_slots(N, V, C) : p.n;
    float2* stats = (float2*)scratch;
    float* target_logit = (float*)((char*)scratch + round256((size_t)slots * N * 8));
    int launches = 0;
    if (bf) {
        HeadEpi e = {};
        e.targets = targets;
        e.stats = stats;
        e.target_logit = target_logit;
        e.vocab = V;
        const int n = launch_head_lse(x, w, N, V, C, e, status, s);
        if (n < 0) return n;
        launches += n;
    } else {
        float* z = (float*)((char*)target_logit + round256((size_t)N * 4));
        for (int i = 0; i < p.n; i++) {
            const int v0 = i * p.width, cols = V - v0 < p.width ? V - v0 : p.width;
            const int n = launch_matmul(dtype, z, 1, x, 0, (const float*)w + (int64_t)v0 * C, 0, nullptr, N, cols, C,
                                        nullptr, status, s);
            if (n < 0) return n;
            piece_stats_kernel<<<(N + 7) / 8, 256, 0, s>>>(stats + (int64_t)i * N, target_logit, z, targets, N, cols,
                                                           v0, V);
            launches += n + 1;
        }
    }
    const int blocks = (N + 31) / 32;
    if (blocks >= 4 * gpt2_num_sms())
        join_kernel<8, 8><<<blocks, 256, 0, s>>>(losses, lse, stats, target_logit, targets, N, V, slots, status);
    else join_kernel<32, 4><<<blocks, 1024, 0, s>>>(losses, lse, stats, target_logit, targets, N, V, slots, status);
    return launches + 1;
}

namespace {

// The matmuls' own scratch (split products), over the pieces.
size_t products_scratch(int N, int C, int V, int dw_fp32, int accumulate, const Pieces& p) {
    size_t most = 0;
    for (int v0 : {0, (p.n - 1) * p.width}) {
        const int cols = round8(V - v0 < p.width ? V - v0 : p.width);
        const size_t a = head_dx_scratch(N, C, cols);
        const size_t b = matmul_scratch(GPT2_MODE_BF16, cols, C, N, dw_fp32, accumulate);
        most = a > most ? a : most;
        most = b > most ? b : most;
    }
    return most;
}

}  // namespace

// A piece of dz; bf16: dx in fp32, the products' own.
size_t linear_classifier_backward_scratch(int dtype, int N, int C, int V, int dw_fp32, int accumulate) {
    const Pieces p = pieces(dtype, N, V);
    if (dtype != GPT2_MODE_BF16) return (size_t)N * p.width * 4;
    return round256((size_t)N * p.width * 2) + round256((size_t)N * C * 4) +
           products_scratch(N, C, V, dw_fp32, accumulate, p);
}

int launch_linear_classifier_backward(int dtype, void* dx, void* dw, int dw_fp32, int accumulate, const void* x,
                                      const void* w, const int32_t* targets, const float* lse, const float* dloss,
                                      const float* dlse, int N, int C, int V, int Vp, void* scratch, int* status,
                                      cudaStream_t s) {
    const bool bf = dtype == GPT2_MODE_BF16;
    const Pieces p = pieces(dtype, N, V);
    int launches = 0;
    const int64_t es = dw_fp32 ? 4 : 2, done = bf ? round8(V) : V;
    if (!accumulate && done < Vp &&
        cudaMemsetAsync((char*)dw + done * C * es, 0, (size_t)(Vp - done) * C * es, s) != cudaSuccess)
        return GPT2_ERR_CUDA;
    if (status) {
        check_targets_kernel<<<(N + 255) / 256, 256, 0, s>>>(targets, N, V, status);
        launches++;
    }
    float* sum = (float*)((char*)scratch + round256((size_t)N * p.width * 2));
    void* own = (char*)sum + round256((size_t)N * C * 4);
    for (int i = 0; i < p.n; i++) {
        const int v0 = i * p.width, cols = V - v0 < p.width ? V - v0 : p.width;
        int n[3] = {0, 0, 0};
        if (bf) {
            const bf16* wp = (const bf16*)w + (int64_t)v0 * C;
            const int pitch = round8(cols);
            HeadEpi e = {};
            e.targets = targets;
            e.lse = lse;
            e.dloss = dloss;
            e.dlse = dlse;
            e.vocab = V;
            e.first = v0;
            n[0] = launch_head_dz(scratch, x, wp, N, pitch, C, cols, e, status, s);
            n[1] = launch_head_dx(sum, scratch, wp, N, C, pitch, cols, i > 0, own, status, s);
            n[2] = launch_matmul(dtype, (char*)dw + (int64_t)v0 * C * es, dw_fp32, scratch, 1, x, 1, nullptr, pitch, C, N,
                                 own, status, s, accumulate);
        } else {
            float* z = (float*)scratch;
            const float* wp = (const float*)w + (int64_t)v0 * C;
            n[0] = launch_matmul(dtype, z, 1, x, 0, wp, 0, nullptr, N, cols, C, nullptr, status, s);
            const int wide = (cols + 255) / 256;
            for (int r0 = 0; r0 < N; r0 += 65535) {
                const int rows = N - r0 < 65535 ? N - r0 : 65535;
                piece_dz_kernel<<<dim3(wide < 64 ? wide : 64, rows), 256, 0, s>>>(
                    z + (int64_t)r0 * cols, targets + r0, lse + r0, dloss ? dloss + r0 : nullptr,
                    dlse ? dlse + r0 : nullptr, rows, cols, v0, V);
                launches++;
            }
            n[1] = launch_matmul(dtype, dx, 1, z, 0, wp, 1, nullptr, N, C, cols, nullptr, status, s, i > 0);
            n[2] = launch_matmul(dtype, (float*)dw + (int64_t)v0 * C, 1, z, 1, x, 1, nullptr, cols, C, N, nullptr, status,
                                 s, accumulate);
        }
        for (int k = 0; k < 3; k++) {
            if (n[k] < 0) return n[k];
            launches += n[k];
        }
    }
    if (bf) {
        const int64_t values = (int64_t)N * C;
        round_kernel<<<(unsigned)((values / 8 + 255) / 256), 256, 0, s>>>((bf16*)dx, sum, values);
        launches++;
    }
    return launches;
}
