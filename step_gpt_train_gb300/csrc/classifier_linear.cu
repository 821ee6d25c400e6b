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
// is fixed). dz is rounded to bf16 for the products, in units of the largest
// |dloss| and |dloss + dlse|, by which the products' sums are scaled in fp32:
// a mean's 1 / n, the same in every row, would otherwise lose up to half a step
// (2^-8) of the whole gradient, in one direction.
//
// fp32: the same with products of fp32 FMA (classifier_linear_f32.cu).
#include "common.cuh"
#include "launch.h"

namespace {

constexpr float LOG2E = 1.4426950408889634f;

// What one piece of dz may take. The gradients of 8192 x 768 x 50257 in pieces of 14592 columns (239 MB) 1337 us, 19456
// 1315, 29184 1295, all at once (824 MB) 1275; of 32768 rows 4096 (268 MB) 5573, 4864 5351, 8192 5363, 12800 (839 MB)
// 5077, 25344 5016, all at once (3.3 GB) 4924: each piece costs its launches, their tails and a pass over dx.
constexpr int64_t PIECE_BYTES = 1ll << 30;
int64_t g_piece_bytes = PIECE_BYTES;  // (linear_classifier_piece() sets it for measurements and tests)

struct Pieces {
    int width, n;
};

// As few pieces as hold at most g_piece_bytes for all rows (or 2048 columns, where that is more), of one width, a whole
// number of tiles. (Widths chosen by a model of the products' rounds of tiles instead, over 13 shapes of 12000 to 65536 rows,
// 256 to 1600 values: between 3.4% faster and 4% slower, the same on average; 32768 x 768 x 50257 5219 us, equal pieces
// 5080.)
Pieces pieces(int dtype, int N, int V) {
    const int64_t es = dtype == GPT2_MODE_BF16 ? 2 : 4;
    int64_t most = g_piece_bytes / ((int64_t)N * es) / 256 * 256;
    if (most < 2048) most = 2048;
    const int n = (int)((V + most - 1) / most), width = ((V + n - 1) / n + 255) / 256 * 256;
    return {width, (V + width - 1) / width};
}
int round8(int v) { return (v + 7) / 8 * 8; }
size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Joins the parts of ROWS rows: strand after strand of slots (neighbouring lanes read neighbouring rows of one slot),
// then the strands. Loads run ahead in batches: a part's exponentials wait for it, the next parts do not. Many rows go
// in blocks of 32 with 8 strands; fewer in blocks of 8 with 64, so that all parts are on their way at once.
template <int ROWS, int STRANDS, int BATCH>
__global__ void __launch_bounds__(STRANDS * ROWS) join_kernel(float* __restrict__ losses, float* __restrict__ lse,
                                                             const float2* __restrict__ stats,
                                                             const float* __restrict__ target_logit,
                                                             const int32_t* __restrict__ targets, int N, int V,
                                                             int slots, int* status) {
    __shared__ float2 sm[STRANDS][ROWS];
    const int tx = threadIdx.x % ROWS, ty = threadIdx.x / ROWS;
    const int64_t row = (int64_t)blockIdx.x * ROWS + tx;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the statistics are still being formed
    float m = -INFINITY, s = 0.f;
    auto join = [&](float2 p) {
        if (p.y == 0.f) return;  // a part without columns
        const float mm = fmaxf(m, p.x);
        s = s * ex2_approx((m - mm) * LOG2E) + p.y * ex2_approx((p.x - mm) * LOG2E);
        m = mm;
    };
    for (int i = ty; i < slots; i += STRANDS * BATCH) {
        float2 p[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; u++) {
            const int slot = i + u * STRANDS;
            p[u] = slot < slots && row < N ? __ldcs(&stats[(int64_t)slot * N + row]) : make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < BATCH; u++) join(p[u]);
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
    const float ls = logf(s), loss = s == 0.f ? INFINITY : (m - target_logit[row]) + ls;  // (0: every logit is -inf)
    lse[row] = m + ls;
    losses[row] = loss < 0.f ? 0.f : loss;
}

// out = in times *scale.
__global__ void __launch_bounds__(256) round_kernel(bf16* __restrict__ out, const float* __restrict__ in, int64_t n,
                                                    const float* __restrict__ scale) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= n) return;
    const float s = *scale;
    float f[8];
    load8_stream(in + i, f);
#pragma unroll
    for (int j = 0; j < 8; j++) f[j] *= s;
    store8(out + i, f);
}

// Targets out of range; and the scale (the largest head_magnitude: 0 where no row counts): by one block as it is, by
// several as float bits (the caller zeroes them), whose largest is the same in any order.
__global__ void __launch_bounds__(1024) rows_kernel(float* __restrict__ scale, const HeadEpi e, int N, int* status) {
    __shared__ float sm[32];
    float m = 0.f;
    bool bad = false;
    for (int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x; i < N; i += (int64_t)gridDim.x * 1024) {
        m = fmaxf(m, head_magnitude(e, i));
        bad |= e.targets[i] < 0 || e.targets[i] >= e.vocab;
    }
    if (bad) set_status(status, GPT2_FLAG_TARGET_RANGE);
    if (!scale) return;
    m = warp_max(m);
    if (threadIdx.x % 32 == 0) sm[threadIdx.x / 32] = m;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    m = warp_max(sm[threadIdx.x]);
    if (threadIdx.x) return;
    if (gridDim.x == 1) *scale = m;
    else atomicMax(reinterpret_cast<unsigned*>(scale), __float_as_uint(m));
}
constexpr int ROWS_A_BLOCK = 32768, FIND_ROWS = 2048;

}  // namespace

void linear_classifier_piece(int64_t bytes) { g_piece_bytes = bytes > 0 ? bytes : PIECE_BYTES; }

// Statistics, target logits.
size_t linear_classifier_forward_scratch(int dtype, int N, int C, int V) {
    const int slots = dtype == GPT2_MODE_BF16 ? head_lse_slots(N, V, C) : head_f32_slots(V);
    return round256((size_t)slots * N * 8) + (size_t)N * 4;
}

int launch_linear_classifier_forward(int dtype, float* losses, float* lse, const void* x, const void* w,
                                     const int32_t* targets, int N, int C, int V, void* scratch, int* status,
                                     cudaStream_t s) {
    const bool bf = dtype == GPT2_MODE_BF16;
    const int slots = bf ? head_lse_slots(N, V, C) : head_f32_slots(V);
    HeadEpi e = {};
    e.targets = targets;
    e.stats = (float2*)scratch;
    e.target_logit = (float*)((char*)scratch + round256((size_t)slots * N * 8));
    e.vocab = V;
    const int n = bf ? launch_head_lse(x, w, N, V, C, e, status, s)
                     : launch_head_f32_lse((const float*)x, (const float*)w, N, V, C, e, s);
    if (n < 0) return n;
    // only its launch overlaps the statistics' kernel: it waits for that one's end (61 rows: 26.3 -> 24.7 us)
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    const float2* stats = e.stats;
    const float* target_logit = e.target_logit;
    cudaError_t r;
    if (N >= 32 * gpt2_num_sms()) {
        cfg.gridDim = (N + 31) / 32;
        cfg.blockDim = 256;
        r = cudaLaunchKernelEx(&cfg, join_kernel<32, 8, 8>, losses, lse, stats, target_logit, targets, N, V, slots, status);
    } else {
        cfg.gridDim = (N + 7) / 8;
        cfg.blockDim = 512;
        r = cudaLaunchKernelEx(&cfg, join_kernel<8, 64, 8>, losses, lse, stats, target_logit, targets, N, V, slots, status);
    }
    if (r != cudaSuccess) return GPT2_ERR_CUDA;
    return n + 1;
}

namespace {

// The columns of dz that a piece's products work on: a multiple of 8; the last piece's go on to dw's last row where its
// buffer has room, so that the rows from V on get their 0 with the others.
int pitch_of(int v0, int V, int Vp, const Pieces& p) {
    const int cols = V - v0 < p.width ? V - v0 : p.width;
    return v0 + p.width >= V && Vp - v0 <= p.width ? Vp - v0 : round8(cols);
}

// The products' own scratch (parts of split products), over the pieces.
size_t products_scratch(int dtype, int N, int C, int V, int Vp, int accumulate, const Pieces& p) {
    const bool bf = dtype == GPT2_MODE_BF16;
    size_t most = 0;
    auto need = [&](size_t n) { most = n > most ? n : most; };
    for (int i = 0; i < p.n; i += p.n > 1 ? p.n - 1 : 1) {
        const int pitch = pitch_of(i * p.width, V, Vp, p);
        if (bf) {
            need(p.n == 1 ? head_scaled_scratch(N, C, pitch, false) : head_dx_scratch(N, C, pitch));
            need(head_scaled_scratch(pitch, C, N, accumulate));
        } else {
            need(head_f32_scratch(N, C, pitch));
            need(head_f32_scratch(pitch, C, N));
        }
    }
    return most;
}

// bf16: the scale; a piece of dz (the first is as wide as any); bf16 in pieces: dx in fp32; the products' own.
struct BackwardScratch {
    size_t dz, dx, own;
    BackwardScratch(int dtype, int N, int C, int V, int Vp, const Pieces& p) {
        const bool bf = dtype == GPT2_MODE_BF16;
        dz = bf ? 256 : 0;
        dx = dz + round256((size_t)N * pitch_of(0, V, Vp, p) * (bf ? 2 : 4));
        own = dx + (bf && p.n > 1 ? round256((size_t)N * C * 4) : 0);
    }
};

}  // namespace

size_t linear_classifier_backward_scratch(int dtype, int N, int C, int V, int Vp, int accumulate) {
    const Pieces p = pieces(dtype, N, V);
    return BackwardScratch(dtype, N, C, V, Vp, p).own + products_scratch(dtype, N, C, V, Vp, accumulate, p);
}

int launch_linear_classifier_backward(int dtype, void* dx, void* dw, int dw_fp32, int accumulate, const void* x,
                                      const void* w, const int32_t* targets, const float* lse, const float* dloss,
                                      const float* dlse, int N, int C, int V, int Vp, void* scratch, int* status,
                                      cudaStream_t s) {
    const bool bf = dtype == GPT2_MODE_BF16;
    const Pieces p = pieces(dtype, N, V);
    const BackwardScratch at(dtype, N, C, V, Vp, p);
    void* dz = (char*)scratch + at.dz;
    float* sum = (float*)((char*)scratch + at.dx);
    void* own = (char*)scratch + at.own;
    int launches = 0;
    const int64_t es = dw_fp32 ? 4 : 2;
    const int last = (p.n - 1) * p.width, done = last + pitch_of(last, V, Vp, p);
    if (!accumulate && done < Vp &&
        cudaMemsetAsync((char*)dw + (int64_t)done * C * es, 0, (size_t)(Vp - done) * C * es, s) != cudaSuccess)
        return GPT2_ERR_CUDA;
    HeadEpi e = {};
    e.targets = targets;
    e.lse = lse;
    e.dloss = dloss;
    e.dlse = dlse;
    e.vocab = V;
    float* scale = e.scale = bf ? (float*)scratch : nullptr;
    // the scale and the targets' check: by the first product's epilogue for few rows (a launch less), else on their own
    const bool find = bf && N <= FIND_ROWS;
    if (!find && (bf || status)) {
        const int blocks = N <= ROWS_A_BLOCK ? 1 : N / ROWS_A_BLOCK < 152 ? N / ROWS_A_BLOCK : 152;
        if (bf && blocks > 1 && cudaMemsetAsync(scale, 0, 4, s) != cudaSuccess) return GPT2_ERR_CUDA;
        rows_kernel<<<blocks, 1024, 0, s>>>(scale, e, N, status);
        launches++;
    }
    for (int i = 0; i < p.n; i++) {
        const int v0 = i * p.width, cols = V - v0 < p.width ? V - v0 : p.width;
        e.first = v0;
        e.find = find && i == 0;
        const int pitch = pitch_of(v0, V, Vp, p);
        int n[3];
        if (bf) {
            const bf16* wp = (const bf16*)w + (int64_t)v0 * C;
            n[0] = launch_head_dz(dz, x, wp, N, pitch, C, cols, e, status, s);
            n[1] = p.n == 1 ? launch_head_dx_scaled(dx, dz, wp, N, C, pitch, cols, scale, own, status, s)
                            : launch_head_dx(sum, dz, wp, N, C, pitch, cols, i > 0, own, status, s);
            n[2] = launch_head_dw((char*)dw + (int64_t)v0 * C * es, dw_fp32, dz, x, pitch, C, N, scale, accumulate, own,
                                  status, s);
        } else {
            const float *xf = (const float*)x, *wp = (const float*)w + (int64_t)v0 * C;
            n[0] = launch_head_f32_dz((float*)dz, xf, wp, N, pitch, C, cols, e, s);
            n[1] = launch_head_f32_dx((float*)dx, (const float*)dz, wp, N, C, pitch, cols, i > 0, own, s);
            n[2] = launch_head_f32_dw((float*)dw + (int64_t)v0 * C, (const float*)dz, xf, pitch, C, N, accumulate, own, s);
        }
        for (int k = 0; k < 3; k++) {
            if (n[k] < 0) return n[k];
            launches += n[k];
        }
    }
    if (bf && p.n > 1) {
        const int64_t values = (int64_t)N * C;
        round_kernel<<<(unsigned)((values / 8 + 255) / 256), 256, 0, s>>>((bf16*)dx, sum, values, scale);
        launches++;
    }
    return launches;
}
