// Norms of queries and keys for each head with the position rotation, in one
// pass, forward and backward (gpt2_op_qk_norm_rotary_*).
//
//   n = x rstd gamma, rstd = 1 / sqrt(mean x^2 + eps)   (or n = x)
//   (y_a, y_b) = amplitude (n_a cos t - n_b sin t, n_a sin t + n_b cos t)
//
// for the pairs (a, b) of the first rot values of a head. The angle t of pair
// j at position p is p * turns[j] in units of 2^-64 turns, modulo one turn: a
// 64-bit product that wraps, so its error does not grow with the position
// (2^-33 of a turn, where a 32-bit product of position and frequency is off by
// 0.006 rad at 10^5); the signed top half, as half turns, goes to sincospif.
//
// A head is held by hd / E neighbouring lanes of a warp, E values (8 or 16
// bytes) each; a warp takes a row and walks its heads, so a lane forms the
// angles of its pairs once a row. The two values of a pair are in one lane
// (interleaved) or in two lanes rot / 2 values apart, which exchange them by a
// shuffle. Every value is read before the lanes of its head write, so the
// output may be the input.
//
// The pass reads and writes each value once: HBM bounds it.
#include "common.cuh"
#include "launch.h"

namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;

// E values of T at p (aligned to their size) as fp32.
__device__ __forceinline__ void load_e(const float* p, float (&f)[4]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
}
__device__ __forceinline__ void load_e(const bf16* p, float (&f)[4]) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    f[0] = __uint_as_float(u.x << 16); f[1] = __uint_as_float(u.x & 0xFFFF0000u);
    f[2] = __uint_as_float(u.y << 16); f[3] = __uint_as_float(u.y & 0xFFFF0000u);
}
template <typename T> __device__ __forceinline__ void load_e(const T* p, float (&f)[8]) { load8(p, f); }
__device__ __forceinline__ void store_e(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store_e(bf16* p, const float (&f)[4]) {
    uint2 u;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
    h[0] = __floats2bfloat162_rn(f[0], f[1]);
    h[1] = __floats2bfloat162_rn(f[2], f[3]);
    *reinterpret_cast<uint2*>(p) = u;
}
template <typename T> __device__ __forceinline__ void store_e(T* p, const float (&f)[8]) { store8(p, f); }

// cos and sin, times the amplitude, of the pairs that this lane's values
// belong to: one for each value in the half layout, one for each two in the
// interleaved one. sin has its sign for this lane's value folded in: the
// rotated value is c * own + s * other.
template <int E, bool PAIRS> struct Angles {
    static constexpr int N = PAIRS ? E / 2 : E;
    float c[N], s[N];

    __device__ __forceinline__ void of(int pos, const uint64_t* turns, int at, int rot, float amplitude) {
        const int half = rot / 2;
#pragma unroll
        for (int i = 0; i < N; i++) {
            int j = PAIRS ? at / 2 + i : at + i;
            if (!PAIRS && j >= half) j -= half;
            c[i] = 1.f;
            s[i] = 0.f;
            if (at < rot) {
                const uint64_t t = (uint64_t)(int64_t)pos * turns[j];
                float sn, cs;
                sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &sn, &cs);
                c[i] = cs * amplitude;
                s[i] = sn * amplitude;
            }
        }
    }
};

// The rotation (dir = 1) or its transpose (dir = -1) of one lane's values. at: the first
// value's place in the head; lanes of one head exchange values by shuffles, so all of a warp call it.
template <int E, bool PAIRS>
__device__ __forceinline__ void rotate(float (&x)[E], const Angles<E, PAIRS>& a, int at, int rot, float dir) {
    if (PAIRS) {
        if (at < rot) {
#pragma unroll
            for (int i = 0; i < E / 2; i++) {
                const float u = x[2 * i], v = x[2 * i + 1], s = dir * a.s[i];
                x[2 * i] = u * a.c[i] - v * s;
                x[2 * i + 1] = u * s + v * a.c[i];
            }
        }
    } else {
        const int half = rot / 2;
        const bool first = at < half;
        const int lane = threadIdx.x & 31;
        // the lane that holds the other values of these pairs
        const int other = at >= rot ? lane : first ? lane + half / E : lane - half / E;
        const float sign = first ? -dir : dir;
#pragma unroll
        for (int i = 0; i < E; i++) {
            const float v = __shfl_sync(0xffffffffu, x[i], other);
            if (at < rot) x[i] = x[i] * a.c[i] + sign * a.s[i] * v;
        }
    }
}

// Sum over the lanes of a head (L a power of two).
template <int L> __device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T, int E, int L, bool PAIRS, bool NORM>
__global__ void __launch_bounds__(THREADS) rotary_forward_kernel(const RotaryArgs a) {
    constexpr int HD = E * L, GROUPS = 32 / L;
    const int lane = threadIdx.x & 31, at = lane % L * E, group = lane / L;
    float gq[E], gk[E];
#pragma unroll
    for (int i = 0; i < E; i++) gq[i] = gk[i] = 1.f;
    if (NORM && a.q_gamma) load_e((const T*)a.q_gamma + at, gq);
    if (NORM && a.k_gamma) load_e((const T*)a.k_gamma + at, gk);
    const int heads = a.Hq + a.Hk;
    for (int64_t row = (int64_t)blockIdx.x * WARPS + threadIdx.x / 32; row < a.N; row += (int64_t)gridDim.x * WARPS) {
        Angles<E, PAIRS> ang;
        ang.of(a.pos[row], a.turns, at, a.rot, a.amplitude);
        const T* q = (const T*)a.q + row * a.q_stride + at;
        const T* k = (const T*)a.k + row * a.k_stride + at;
        T* qo = (T*)a.qo + row * a.qo_stride + at;
        T* ko = (T*)a.ko + row * a.ko_stride + at;
#pragma unroll 4
        for (int h0 = 0; h0 < heads; h0 += GROUPS) {
            const int h = h0 + group;
            const bool key = h >= a.Hq;
            float x[E];
#pragma unroll
            for (int i = 0; i < E; i++) x[i] = 0.f;
            if (h < heads) load_e(key ? k + (h - a.Hq) * HD : q + h * HD, x);
            if (NORM) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < E; i++) ss += x[i] * x[i];
                const float r = 1.f / sqrtf(head_sum<L>(ss) * (1.f / HD) + a.eps);
#pragma unroll
                for (int i = 0; i < E; i++) x[i] *= r * (key ? gk[i] : gq[i]);
            }
            rotate<E, PAIRS>(x, ang, at, a.rot, 1.f);
            if (h < heads) store_e(key ? ko + (h - a.Hq) * HD : qo + h * HD, x);
        }
    }
}

// With dn the gradient turned back and xhat = x rstd: dgamma = sum dn xhat,
// dx = rstd (dn gamma - xhat mean(dn gamma xhat)). A lane's values lie at the
// same place of every head it sees, so it keeps its share of dgamma in
// registers over all its rows; block sums go to partial [block][2][HD], which
// a column sum adds in a fixed order.
template <typename T, int E, int L, bool PAIRS, bool NORM>
__global__ void __launch_bounds__(THREADS) rotary_backward_kernel(const RotaryArgs a, float* __restrict__ partial) {
    constexpr int HD = E * L, GROUPS = 32 / L;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, at = lane % L * E, group = lane / L;
    float gq[E], gk[E], aq[E], ak[E];
#pragma unroll
    for (int i = 0; i < E; i++) {
        gq[i] = gk[i] = 1.f;
        aq[i] = ak[i] = 0.f;
    }
    if (NORM && a.q_gamma) load_e((const T*)a.q_gamma + at, gq);
    if (NORM && a.k_gamma) load_e((const T*)a.k_gamma + at, gk);
    for (int64_t row = (int64_t)blockIdx.x * WARPS + warp; row < a.N; row += (int64_t)gridDim.x * WARPS) {
        Angles<E, PAIRS> ang;
        ang.of(a.pos[row], a.turns, at, a.rot, a.amplitude);
        auto heads = [&](int H, const T* dy, const T* x, T* dx, const float (&gamma)[E], float (&acc)[E]) {
#pragma unroll 2
            for (int h0 = 0; h0 < H; h0 += GROUPS) {
                const int h = h0 + group;
                float d[E], v[E];
#pragma unroll
                for (int i = 0; i < E; i++) d[i] = v[i] = 0.f;
                if (h < H) {
                    load_e(dy + h * HD, d);
                    if (NORM) load_e(x + h * HD, v);
                }
                rotate<E, PAIRS>(d, ang, at, a.rot, -1.f);
                if (NORM) {
                    float ss = 0.f, in = 0.f;
#pragma unroll
                    for (int i = 0; i < E; i++) ss += v[i] * v[i];
                    const float r = 1.f / sqrtf(head_sum<L>(ss) * (1.f / HD) + a.eps);
#pragma unroll
                    for (int i = 0; i < E; i++) {
                        v[i] *= r;
                        acc[i] += d[i] * v[i];
                        d[i] *= gamma[i];
                        in += d[i] * v[i];
                    }
                    in = head_sum<L>(in) * (1.f / HD);
#pragma unroll
                    for (int i = 0; i < E; i++) d[i] = r * (d[i] - v[i] * in);
                }
                if (h < H) store_e(dx + h * HD, d);
            }
        };
        heads(a.Hq, (const T*)a.dqo + row * a.dqo_stride + at, (const T*)a.q + row * a.q_stride + at,
              (T*)a.qo + row * a.qo_stride + at, gq, aq);
        heads(a.Hk, (const T*)a.dko + row * a.dko_stride + at, (const T*)a.k + row * a.k_stride + at,
              (T*)a.ko + row * a.ko_stride + at, gk, ak);
    }
    if constexpr (NORM) {
    if (!partial) return;
    __shared__ float sm[WARPS][2][HD];
#pragma unroll
    for (int i = 0; i < E; i++) {
#pragma unroll
        for (int o = L; o < 32; o <<= 1) {
            aq[i] += __shfl_xor_sync(0xffffffffu, aq[i], o);
            ak[i] += __shfl_xor_sync(0xffffffffu, ak[i], o);
        }
        if (group == 0) {
            sm[warp][0][at + i] = aq[i];
            sm[warp][1][at + i] = ak[i];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * HD; c += THREADS) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; w++) t += sm[w][c / HD][c % HD];
        partial[(int64_t)blockIdx.x * 2 * HD + c] = t;
    }
    }
}

int rotary_blocks(int N) {
    const int64_t rows = ((int64_t)N + WARPS - 1) / WARPS, most = (int64_t)gpt2_num_sms() * 8;
    return (int)(rows < most ? rows : most);
}

template <typename T, int E, int L, bool PAIRS, bool NORM>
int start(const RotaryArgs& a, bool back, float* partial, cudaStream_t s) {
    const int blocks = rotary_blocks(a.N);
    if (back) rotary_backward_kernel<T, E, L, PAIRS, NORM><<<blocks, THREADS, 0, s>>>(a, partial);
    else rotary_forward_kernel<T, E, L, PAIRS, NORM><<<blocks, THREADS, 0, s>>>(a);
    return blocks;
}

template <typename T, int E, int L>
int start(const RotaryArgs& a, bool back, float* partial, cudaStream_t s) {
    if (a.interleaved)
        return a.norm ? start<T, E, L, true, true>(a, back, partial, s) : start<T, E, L, true, false>(a, back, partial, s);
    return a.norm ? start<T, E, L, false, true>(a, back, partial, s) : start<T, E, L, false, false>(a, back, partial, s);
}

template <typename T>
int start(const RotaryArgs& a, bool back, float* partial, cudaStream_t s) {
    switch (a.hd) {
        case 8: return start<T, 4, 2>(a, back, partial, s);
        case 16: return start<T, 4, 4>(a, back, partial, s);
        case 32: return start<T, 4, 8>(a, back, partial, s);
        case 64: return start<T, 4, 16>(a, back, partial, s);
        default: return start<T, 4, 32>(a, back, partial, s);
    }
}

}  // namespace

size_t rotary_backward_scratch(int N, int hd) { return (size_t)rotary_blocks(N) * 2 * hd * 4; }

int launch_rotary(int dtype, const RotaryArgs& a, bool back, float* dq_gamma, float* dk_gamma, void* scratch,
                  cudaStream_t s) {
    float* partial = back && a.norm && (dq_gamma || dk_gamma) ? (float*)scratch : nullptr;
    const int blocks = dtype == GPT2_MODE_BF16 ? start<bf16>(a, back, partial, s) : start<float>(a, back, partial, s);
    if (!partial) return 1;
    ColsumJob job = {partial, {dq_gamma, dk_gamma, nullptr}, blocks, 2 * a.hd, a.hd, 0};
    return 1 + launch_colsum_jobs(&job, 1, s);
}
