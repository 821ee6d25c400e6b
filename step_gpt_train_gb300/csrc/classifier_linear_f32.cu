// The linear classifier's products in fp32 (exact-parity mode: fp32 FMA, no
// reduced precision): x W^T reduced to row statistics or turned into dz, and
// the two products that read dz (classifier_linear.cu).
//
// 64 x 64 tiles, 128 threads of 8 x 4 outputs. Both operands lie in shared
// memory with k innermost, 16 of it and 4 of padding: a thread's rows are 8
// apart and its columns 16 apart, so that a warp's 16-byte reads meet different
// banks. Two neighbouring k's of a row are one register pair, and the paired
// FMA keeps a sum over the even and one over the odd k's: half the instructions
// of single FMAs, no operand to duplicate, and sums of half the length. Slices
// are under way two or three ahead: [rows][k] operands by asynchronous copies,
// [k][rows] ones through registers, which turn them. Products with few tiles
// (dx: N x C outputs, K = V) are cut along k; a second kernel adds the parts in
// order.
//
// 1021 x 128 x 5003 (1.3 GFLOP a product, 17 us at 75 TFLOP/s): TIMES
#include "common.cuh"
#include "launch.h"
#include "tc_common.cuh"

namespace {

using tc::f2_fma;
using tc::f2_pack;
using tc::f2_unpack;

constexpr int T = 64, KS = 16, PITCH = KS + 4, THREADS = 128;
constexpr int TM = 8, TN = 4;

constexpr int STORE = 0, LSE = 1, DZ = 2;

// Rows, columns and k's are multiples of 4 where vectors run along them (x, w and dz are so laid out).
struct Product {
    const float *A, *B;
    float* D;          // STORE: [M][N], or the parts [split][M][N]; DZ: [M][N]
    int M, N, K;
    int b_rows;        // the rows of B that are read (n's, or k's where B is [k][n]); the rest count as 0
    int per_split;     // k's of a part, a multiple of KS
    int accumulate;    // STORE without parts: D +=
    HeadEpi head;
};

// Where a row keeps its k's in shared memory: its four vectors in an order that changes every 8 rows. A warp that stores
// [k][rows] data writes one value to each of 16 rows 4 apart, 80 words from one to the next: in one order they would meet
// two banks, in this one eight.
__device__ __forceinline__ constexpr int place(int row, int k) { return (((k >> 2) ^ (row >> 3)) & 3) * 4 + (k & 3); }

// A slice of an operand: T rows by KS k's from (row0, k0), two vectors of four a thread; zeros outside `rows` and k1.
// [rows][k]: copied as it is.
__device__ __forceinline__ void copy_slice(float (*s)[PITCH], const float* p, int rows, int K, int row0, int k0, int k1) {
#pragma unroll
    for (int u = 0; u < 2; u++) {
        const int i = threadIdx.x + u * THREADS, r = row0 + i / 4, k = k0 + i % 4 * 4;
        const bool in = r < rows && k < k1;
        const float* from = in ? p + (int64_t)r * K + k : p;
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(&s[i / 4][place(i / 4, i % 4 * 4)]);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
    }
}
// [k][rows]: through registers, turned when stored.
struct Turned {
    float f[2][4];
    __device__ __forceinline__ void load(const float* p, int rows, int row0, int k0, int k1) {
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const int i = threadIdx.x + u * THREADS, r = row0 + i % 16 * 4, k = k0 + i / 16;
            const float4 v = r < rows && k < k1 ? *reinterpret_cast<const float4*>(p + (int64_t)k * rows + r)
                                                : make_float4(0.f, 0.f, 0.f, 0.f);
            f[u][0] = v.x, f[u][1] = v.y, f[u][2] = v.z, f[u][3] = v.w;
        }
    }
    __device__ __forceinline__ void store(float (*s)[PITCH]) const {
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const int i = threadIdx.x + u * THREADS;
#pragma unroll
            for (int j = 0; j < 4; j++) s[i % 16 * 4 + j][place(i % 16 * 4, i / 16)] = f[u][j];
        }
    }
};

template <bool A_MN, bool B_MN, int EPI>
__global__ void __launch_bounds__(THREADS, 3) head_f32_kernel(const Product g) {
    constexpr int STAGES = A_MN || B_MN ? 3 : 4, AHEAD = STAGES - 1;
    __shared__ __align__(16) float As[STAGES][T][PITCH], Bs[STAGES][T][PITCH];
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const int n_tiles = (g.N + T - 1) / T;
    const int m0 = blockIdx.x / n_tiles * T, n0 = blockIdx.x % n_tiles * T;
    const int k0 = blockIdx.y * g.per_split, k1 = min(g.K, k0 + g.per_split);
    uint64_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) acc[i][j] = 0;
    // A slice goes to its stage AHEAD slices early if it is copied; a turned one is loaded two slices early and stored
    // one early (a stage was last read two slices before that, and there is a barrier between).
    auto copy = [&](int k, int stage) {
        if (!A_MN) copy_slice(As[stage], g.A, g.M, g.K, m0, k, k1);
        if (!B_MN) copy_slice(Bs[stage], g.B, g.b_rows, g.K, n0, k, k1);
        cp_async_commit();
    };
    Turned a, b;
    auto load = [&](int k) {
        if (A_MN) a.load(g.A, g.M, m0, k, k1);
        if (B_MN) b.load(g.B, g.N, n0, k, min(k1, g.b_rows));
    };
    auto store = [&](int stage) {
        if (A_MN) a.store(As[stage]);
        if (B_MN) b.store(Bs[stage]);
    };
#pragma unroll
    for (int u = 0; u < AHEAD; u++) copy(k0 + u * KS, u);
    load(k0);
    store(0);
    load(k0 + KS);
    int stage = 0;
    auto after = [&](int n) { return stage + n >= STAGES ? stage + n - STAGES : stage + n; };
    for (int k = k0; k < k1; k += KS) {
        cp_async_wait<AHEAD - 1>();
        __syncthreads();
        copy(k + AHEAD * KS, after(AHEAD));
        store(after(1));
        load(k + 2 * KS);
#pragma unroll
        for (int kk = 0; kk < KS; kk += 4) {
            ulonglong2 x[TM], y[TN];
#pragma unroll
            for (int i = 0; i < TM; i++) x[i] = *reinterpret_cast<const ulonglong2*>(&As[stage][ty + 8 * i][place(8 * i, kk)]);
#pragma unroll
            for (int j = 0; j < TN; j++)
                y[j] = *reinterpret_cast<const ulonglong2*>(&Bs[stage][tx + 16 * j][place(tx + 16 * j, kk)]);
#pragma unroll
            for (int i = 0; i < TM; i++)
#pragma unroll
                for (int j = 0; j < TN; j++) acc[i][j] = f2_fma(x[i].x, y[j].x, acc[i][j]);
#pragma unroll
            for (int i = 0; i < TM; i++)
#pragma unroll
                for (int j = 0; j < TN; j++) acc[i][j] = f2_fma(x[i].y, y[j].y, acc[i][j]);
        }
        stage = after(1);
    }
    float* d = g.D + (EPI == STORE ? (int64_t)blockIdx.y * g.M * g.N : 0);
#pragma unroll
    for (int i = 0; i < TM; i++) {
        const int row = m0 + ty + 8 * i;  // the same for the 16 lanes of a half warp
        float z[TN];
#pragma unroll
        for (int j = 0; j < TN; j++) {
            float lo, hi;
            f2_unpack(acc[i][j], lo, hi);
            z[j] = lo + hi;
        }
        if (EPI == STORE) {
            if (row >= g.M) continue;
#pragma unroll
            for (int j = 0; j < TN; j++) {
                const int n = n0 + tx + 16 * j;
                if (n < g.N) {
                    float* p = d + (int64_t)row * g.N + n;
                    *p = g.accumulate ? *p + z[j] : z[j];
                }
            }
            continue;
        }
        int t = -1;
        if (row < g.M) {
            t = g.head.targets[row];
            if (t < 0 || t >= g.head.vocab) t = 0;
            t -= g.head.first;
        }
        if (EPI == LSE) {
            float m = -INFINITY, s = 0.f;
#pragma unroll
            for (int j = 0; j < TN; j++)
                if (n0 + tx + 16 * j < g.N) m = fmaxf(m, z[j]);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
            for (int j = 0; j < TN; j++) {
                const int n = n0 + tx + 16 * j;
                if (n < g.N) s += expf(z[j] - (m > -INFINITY ? m : 0.f));  // (nothing but -inf: 0; a NaN stays)
                if (n == t && row < g.M) g.head.target_logit[row] = z[j];
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (tx == 0 && row < g.M) g.head.stats[(int64_t)(n0 / T) * g.M + row] = make_float2(m, s);
        } else if (row < g.M) {
            const float dl = g.head.dloss ? g.head.dloss[row] : 0.f;
            const float w = dl + (g.head.dlse ? g.head.dlse[row] : 0.f), l = g.head.lse[row];
            const bool counts = (w != 0.f || dl != 0.f) && l != -INFINITY;
#pragma unroll
            for (int j = 0; j < TN; j++) {
                const int n = n0 + tx + 16 * j;
                // a row that does not count gets zeros whatever its logits are
                if (n < g.N) d[(int64_t)row * g.N + n] = counts && n < g.b_rows ? w * expf(z[j] - l) - (n == t ? dl : 0.f) : 0.f;
            }
        }
    }
}

// D = or += the parts, added in order.
__global__ void __launch_bounds__(256) head_f32_join_kernel(float* __restrict__ D, const float* __restrict__ parts,
                                                            int64_t n, int splits, int accumulate) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float s = 0.f;
#pragma unroll 4
    for (int k = 0; k < splits; k++) s += parts[k * n + i];
    D[i] = accumulate ? D[i] + s : s;
}

int64_t tiles(int M, int N) { return (int64_t)((M + T - 1) / T) * ((N + T - 1) / T); }

// Parts of k: as many as fill the device's three blocks an SM, of at least 256 k's each.
int splits(int M, int N, int K) {
    const int64_t room = (int64_t)gpt2_num_sms() * 3 / tiles(M, N), most = K / 256;
    const int64_t s = room < most ? room : most;
    return s < 1 ? 1 : (int)s;
}

template <bool A_MN, bool B_MN>
int start_store(float* D, const float* A, const float* B, int M, int N, int K, int b_rows, bool accumulate,
                float* scratch, cudaStream_t s) {
    const int sp = splits(M, N, K);
    Product g = {};
    g.A = A, g.B = B, g.M = M, g.N = N, g.K = K, g.b_rows = b_rows;
    g.per_split = ((K + sp - 1) / sp + KS - 1) / KS * KS;
    const int parts = (K + g.per_split - 1) / g.per_split;
    g.D = parts > 1 ? scratch : D;
    g.accumulate = parts == 1 && accumulate;
    head_f32_kernel<A_MN, B_MN, STORE><<<dim3((unsigned)tiles(M, N), parts), THREADS, 0, s>>>(g);
    if (parts == 1) return 1;
    const int64_t n = (int64_t)M * N;
    head_f32_join_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(D, scratch, n, parts, accumulate);
    return 2;
}

template <int EPI>
int start_head(float* D, const float* x, const float* w, int M, int N, int K, int b_rows, const HeadEpi& e,
               cudaStream_t s) {
    Product g = {};
    g.A = x, g.B = w, g.D = D, g.M = M, g.N = N, g.K = K, g.b_rows = b_rows, g.per_split = (K + KS - 1) / KS * KS;
    g.head = e;
    head_f32_kernel<false, false, EPI><<<(unsigned)tiles(M, N), THREADS, 0, s>>>(g);
    return 1;
}

}  // namespace

int head_f32_slots(int V) { return (V + T - 1) / T; }

int launch_head_f32_lse(const float* x, const float* w, int M, int N, int K, const HeadEpi& e, cudaStream_t s) {
    return start_head<LSE>(nullptr, x, w, M, N, K, N, e, s);
}
int launch_head_f32_dz(float* dz, const float* x, const float* w, int M, int N, int K, int rows, const HeadEpi& e,
                       cudaStream_t s) {
    return start_head<DZ>(dz, x, w, M, N, K, rows, e, s);
}
size_t head_f32_scratch(int M, int N, int K) {
    const int sp = splits(M, N, K);
    return sp > 1 ? (size_t)sp * M * N * 4 : 0;
}
int launch_head_f32_dx(float* dx, const float* dz, const float* w, int M, int N, int K, int rows, bool add, void* scratch,
                       cudaStream_t s) {
    return start_store<false, true>(dx, dz, w, M, N, K, rows, add, (float*)scratch, s);
}
int launch_head_f32_dw(float* dw, const float* dz, const float* x, int M, int N, int K, bool add, void* scratch,
                       cudaStream_t s) {
    return start_store<true, true>(dw, dz, x, M, N, K, K, add, (float*)scratch, s);
}
