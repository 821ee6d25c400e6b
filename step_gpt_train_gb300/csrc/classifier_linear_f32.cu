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
// 1021 x 128 x 5003 (1.3 GFLOP a product, 17 us at 75 TFLOP/s): dz 44 us, dx 34
// and dw 47, and 3 each to add their parts. What bounds it: three blocks of 160
// registers an SM are at most three warps to a scheduler, and 27% (dw, 316 blocks
// for 456 places) to 41% (dz) of the issue slots are used. Between two of a warp's
// instructions lie 1.0 to 1.4 cycles of fixed latencies, 0.5 to 0.9 of waiting for
// the FMA pipe and 0.4 to 0.5 for operands from shared memory; a third of what is
// issued is not FMA.
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

// A thread's two vectors of four of each slice (T rows by KS k's) of an operand, walked along k; zeros outside `rows`
// and k1. [rows][k]: copied as they are.
struct Copied {
    const float* from[2];
    uint32_t to[2];
    int k, k1;
    bool in[2];
    __device__ __forceinline__ Copied(const float* p, int rows, int K, int row0, int k0, int k1_, float (*s)[PITCH])
        : k(k0 + threadIdx.x % 4 * 4), k1(k1_) {
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const int r = threadIdx.x / 4 + u * (THREADS / 4);
            in[u] = row0 + r < rows;
            from[u] = p + (in[u] ? (int64_t)(row0 + r) * K + k : 0);
            to[u] = (uint32_t)__cvta_generic_to_shared(&s[r][place(r, threadIdx.x % 4 * 4)]);
        }
    }
    __device__ __forceinline__ void next(int stage) {
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const bool now = in[u] && k < k1;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to[u] + stage * (T * PITCH * 4)),
                         "l"(now ? from[u] : from[u] - (in[u] ? k : 0)), "r"(now ? 16 : 0)
                         : "memory");
            if (in[u]) from[u] += KS;
        }
        k += KS;
    }
};
// [k][rows]: through registers, turned when stored.
struct Turned {
    float f[2][4];
    const float* from[2];
    int64_t step;
    int k, k1;
    bool in;
    __device__ __forceinline__ Turned(const float* p, int rows, int row0, int k0, int k1_) : k(k0 + threadIdx.x / 16), k1(k1_) {
        const int r = row0 + threadIdx.x % 16 * 4;
        in = r < rows;
        step = (int64_t)KS * rows;
#pragma unroll
        for (int u = 0; u < 2; u++) from[u] = p + (int64_t)(k + u * (THREADS / 16)) * rows + r;
    }
    __device__ __forceinline__ void next() {
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const float4 v = in && k + u * (THREADS / 16) < k1 ? *reinterpret_cast<const float4*>(from[u])
                                                              : make_float4(0.f, 0.f, 0.f, 0.f);
            f[u][0] = v.x, f[u][1] = v.y, f[u][2] = v.z, f[u][3] = v.w;
            from[u] += step;
        }
        k += KS;
    }
    __device__ __forceinline__ void store(float (*s)[PITCH]) const {
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
            for (int j = 0; j < 4; j++)
                s[threadIdx.x % 16 * 4 + j][place(threadIdx.x % 16 * 4, threadIdx.x / 16 + u * (THREADS / 16))] = f[u][j];
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
    Copied ca(g.A, A_MN ? 0 : g.M, g.K, m0, k0, k1, As[0]), cb(g.B, B_MN ? 0 : g.b_rows, g.K, n0, k0, k1, Bs[0]);
    Turned ta(g.A, A_MN ? g.M : 0, m0, k0, k1), tb(g.B, B_MN ? g.N : 0, n0, k0, min(k1, g.b_rows));
    auto copy = [&](int stage) {
        if (!A_MN) ca.next(stage);
        if (!B_MN) cb.next(stage);
        cp_async_commit();
    };
    auto load = [&]() {
        if (A_MN) ta.next();
        if (B_MN) tb.next();
    };
    auto store = [&](int stage) {
        if (A_MN) ta.store(As[stage]);
        if (B_MN) tb.store(Bs[stage]);
    };
#pragma unroll
    for (int u = 0; u < AHEAD; u++) copy(u);
    load();
    store(0);
    load();
    int stage = 0;
    auto after = [&](int n) { return stage + n >= STAGES ? stage + n - STAGES : stage + n; };
    // place(8 i, kk) is a constant; place(tx + 16 j, kk) exchanges neighbouring vectors for tx >= 8: from two bases,
    // one for even and one for odd vectors, its places are constants too
    const int turn = (tx >> 3) * 4;
    for (int k = k0; k < k1; k += KS) {
        cp_async_wait<AHEAD - 1>();
        __syncthreads();
        copy(after(AHEAD));
        store(after(1));
        load();
        const float *pa = &As[stage][ty][0], *pe = &Bs[stage][tx][0] + turn, *po = &Bs[stage][tx][0] - turn;
#pragma unroll
        for (int q = 0; q < KS / 4; q++) {
            ulonglong2 x[TM], y[TN];
#pragma unroll
            for (int i = 0; i < TM; i++) x[i] = *reinterpret_cast<const ulonglong2*>(pa + 8 * i * PITCH + place(8 * i, 4 * q));
#pragma unroll
            for (int j = 0; j < TN; j++) {
                const int c = place(16 * j, 4 * q);  // of tx < 8
                y[j] = *reinterpret_cast<const ulonglong2*>((c & 4 ? po : pe) + 16 * j * PITCH + c);
            }
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
