// Norms of queries and keys for each head with the position rotation, in one
// pass, forward and backward (gpt2_op_qk_norm_rotary_*).
//
//   n = x rstd gamma, rstd = 1 / sqrt(mean x^2 + eps)   (or n = x)
//   (y_a, y_b) = amplitude (n_a cos t - n_b sin t, n_a sin t + n_b cos t)
//
// for the pairs (a, b) of the first rot values of a head. The angle t of pair
// j at position p is p * turns[j] in units of 2^-64 turns, modulo one turn: a
// 64-bit product that wraps, whose error is the table's alone (2^-34 of a turn
// at position 2^31, where a 32-bit product of position and frequency is off by
// 0.006 rad at 10^5). The nearest quarter turn is taken off in whole numbers; what
// is left, an eighth of a turn at most, is rounded to fp32 (2^-28 of a turn) for
// sincospif, and the quarters exchange cos and sin and turn their signs.
//
// A head is held by hd / E neighbouring lanes of a warp, E values (16 bytes, or
// 8 where the halves of a pair would not lie in whole lanes) each. A warp takes
// a row: its lanes form the angles of the row's pairs once, share them through
// shared memory, and walk the heads, a few of them loaded at a time. The two
// values of a pair are in one lane (interleaved) or in two lanes rot / 2 values
// apart, which exchange them by shuffles. Every value is read before the lanes
// of its head write, so the output may be the input.
//
// The pass reads and writes each value once: HBM bounds it where the
// instructions of a value (an unpacking, a square, three products, an exchange,
// a packing; on pairs of values where they lie so) leave it room.
#include "common.cuh"
#include "launch.h"
#include "tc_common.cuh"

namespace {

using tc::f2_fma;
using tc::f2_mul;
using tc::f2_pack;
using tc::f2_unpack;

// A block's warps, the blocks on an SM and the steps whose copies are in flight. At 32768 rows of 24 heads of 64
// (bf16, with norms): three blocks of the forward 37.3 us, two 41.0, four 41.0 (64 registers: spills); two blocks of
// the backward 54.4, one 69.7, three 63.3 (80 registers). From two steps ahead to eight: within 1 us. (Measured before
// the angles left their quarter turns in whole numbers: in one loop of both, 36.95 -> 37.05 and 57.15 -> 57.7.)
constexpr int WARPS = 8;
constexpr int FORWARD_A_SM = 3, BACKWARD_A_SM = 2;
constexpr int AHEAD = 4;
constexpr int MOST_PAIRS = 64;

// E values of T as loaded, and as fp32.
template <typename T, int E> struct Raw;
template <> struct __align__(16) Raw<bf16, 8> { uint32_t w[4]; };
template <> struct __align__(8) Raw<bf16, 4> { uint32_t w[2]; };
template <> struct __align__(16) Raw<float, 4> { uint32_t w[4]; };

template <int E> __device__ __forceinline__ void unpack(const Raw<bf16, E>& r, float (&f)[E]) {
#pragma unroll
    for (int i = 0; i < E / 2; i++) {
        f[2 * i] = __uint_as_float(r.w[i] << 16);
        f[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const Raw<float, 4>& r, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; i++) f[i] = __uint_as_float(r.w[i]);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store_e(bf16* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ void store_e(bf16* p, const float (&f)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
}
__device__ __forceinline__ void store_e(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}

// x *= y, and the sum of x y, on pairs of values.
template <int E> __device__ __forceinline__ void times(float (&x)[E], const float (&y)[E]) {
#pragma unroll
    for (int i = 0; i < E; i += 2)
        f2_unpack(f2_mul(f2_pack(x[i], x[i + 1]), f2_pack(y[i], y[i + 1])), x[i], x[i + 1]);
}
template <int E> __device__ __forceinline__ void times(float (&x)[E], float y) {
    const uint64_t yy = f2_pack(y, y);
#pragma unroll
    for (int i = 0; i < E; i += 2) f2_unpack(f2_mul(f2_pack(x[i], x[i + 1]), yy), x[i], x[i + 1]);
}
template <int E> __device__ __forceinline__ float dot(const float (&x)[E], const float (&y)[E]) {
    uint64_t s = f2_mul(f2_pack(x[0], x[1]), f2_pack(y[0], y[1]));
#pragma unroll
    for (int i = 2; i < E; i += 2) s = f2_fma(f2_pack(x[i], x[i + 1]), f2_pack(y[i], y[i + 1]), s);
    float a, b;
    f2_unpack(s, a, b);
    return a + b;
}
// Sum over the lanes of a head (L a power of two).
template <int L> __device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A warp's cos, sin and -sin of a row's pairs, times the amplitude, and behind them 1 and 0 for values that are not
// rotated.
struct Shared {
    __align__(16) float cos[MOST_PAIRS + 8], sin[2][MOST_PAIRS + 8];
};

template <int N> __device__ __forceinline__ void load_shared(float (&f)[N], const float* p) {
    if (N == 2) {
        const float2 v = *reinterpret_cast<const float2*>(p);
        f[0] = v.x, f[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + i);
            f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
        }
    }
}

// Those of the pairs that this lane's values belong to: one for each value in the half layout (sin with the sign that
// turns the other value into this one's share: y = c x + s x_other), one for each two in the interleaved one.
template <int E, bool PAIRS> struct Angles {
    static constexpr int N = PAIRS ? E / 2 : E;
    float c[N], s[N];

    static __device__ __forceinline__ void begin(Shared& w) {
        const int lane = threadIdx.x & 31;
        if (lane < 8) {
            w.cos[MOST_PAIRS + lane] = 1.f;
            w.sin[0][MOST_PAIRS + lane] = w.sin[1][MOST_PAIRS + lane] = 0.f;
        }
    }
    __device__ __forceinline__ void of(int pos, const uint64_t* turns, int at, int rot, float amplitude, Shared& w) {
        const int half = rot / 2, lane = threadIdx.x & 31;
        __syncwarp();  // the row before has read its angles
        for (int j = lane; j < half; j += 32) {
            const uint64_t t = (uint64_t)(int64_t)pos * turns[j];
            const uint32_t quarter = (uint32_t)((t + (1ull << 61)) >> 62);
            float sn, cs;
            // (32 bits, to 2^-34 of a turn, are converted in less time than 64)
            sincospif((float)(int32_t)((t - ((uint64_t)quarter << 62)) >> 30) * 0x1p-33f, &sn, &cs);
            if (quarter & 1) {
                const float c = cs;
                cs = -sn;
                sn = c;
            }
            if (quarter & 2) {
                cs = -cs;
                sn = -sn;
            }
            w.cos[j] = cs * amplitude;
            w.sin[0][j] = sn * amplitude;
            w.sin[1][j] = -sn * amplitude;
        }
        __syncwarp();
        const bool first = !PAIRS && at < half;
        const int j0 = at >= rot ? MOST_PAIRS : PAIRS ? at / 2 : first ? at : at - half;
        load_shared(c, w.cos + j0);
        load_shared(s, w.sin[first] + j0);
    }
};

// The rotation of one lane's values, or its transpose (BACK). other: the lane that holds the other values of
// its pairs (half layout). Lanes of a head exchange values, so all of a warp call it.
template <int E, bool PAIRS, bool BACK>
__device__ __forceinline__ void rotate(float (&x)[E], const Angles<E, PAIRS>& a, int other) {
    if (PAIRS) {
#pragma unroll
        for (int i = 0; i < E / 2; i++) {
            const float u = x[2 * i], v = x[2 * i + 1], s = BACK ? -a.s[i] : a.s[i];
            x[2 * i] = u * a.c[i] - v * s;
            x[2 * i + 1] = u * s + v * a.c[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const float v = __shfl_sync(0xffffffffu, x[i], other), w = __shfl_sync(0xffffffffu, x[i + 1], other);
            const uint64_t s = BACK ? f2_pack(-a.s[i], -a.s[i + 1]) : f2_pack(a.s[i], a.s[i + 1]);
            const uint64_t y = f2_mul(f2_pack(v, w), s);
            f2_unpack(f2_fma(f2_pack(x[i], x[i + 1]), f2_pack(a.c[i], a.c[i + 1]), y), x[i], x[i + 1]);
        }
    }
}

// This lane's place in its head (at), its head among the warp's (group), and its partner for the half layout.
template <int E, int L> struct Place {
    int lane, at, group, other;
    __device__ __forceinline__ explicit Place(int rot) {
        lane = threadIdx.x & 31;
        at = lane % L * E;
        group = lane / L;
        other = at >= rot ? lane : at < rot / 2 ? lane + rot / 2 / E : lane - rot / 2 / E;
    }
};

// The norms' weights in fp32 (ones where there are none), for a block.
template <typename T, int HD>
__device__ __forceinline__ void load_weights(float (&w)[2][HD], const void* q_gamma, const void* k_gamma) {
    for (int i = threadIdx.x; i < 2 * HD; i += WARPS * 32) {
        const T* g = (const T*)(i < HD ? q_gamma : k_gamma);
        w[i / HD][i % HD] = g ? to_float(g[i % HD]) : 1.f;
    }
}

// What a warp walks: its rows, and in each the query heads and then the key heads, a step of GROUPS heads at a time.
// Sources of one kind (values, or gradients) by their rows' places.
template <typename T> struct Source {
    const T *q, *k;
    int64_t q_step, k_step;
    __device__ __forceinline__ Source(const void* q0, int64_t q_stride, const void* k0, int64_t k_stride, int64_t row, int at)
        : q((const T*)q0 + row * q_stride + at), k((const T*)k0 + row * k_stride + at),
          q_step(q_stride * (int64_t)(gridDim.x * WARPS)), k_step(k_stride * (int64_t)(gridDim.x * WARPS)) {}
    __device__ __forceinline__ void next() { q += q_step, k += k_step; }
};

// A lane's vectors of the next DEPTH steps, on their way to its own slots of shared memory: the copies hold no
// registers, so they run as far ahead as HBM needs them to. A lane reads what it copied itself, so it waits for its
// own copies only. One slot more than copies in flight: the slot that a copy goes to was read a step ago.
template <typename T, int E, int DEPTH, int SOURCES> struct Ring {
    static constexpr int BYTES = E * sizeof(T);
    static constexpr int SLOTS = DEPTH + 1;
    char* mine;  // [SLOTS][SOURCES], 32 lanes' vectors apart
    int at;

    __device__ __forceinline__ void copy(int slot, int source, const T* from) {
        const uint32_t s = (uint32_t)__cvta_generic_to_shared(mine + (slot * SOURCES + source) * 32 * BYTES);
        if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(from) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(s), "l"(from) : "memory");
    }
    __device__ __forceinline__ Raw<T, E> read(int source) const {
        return *reinterpret_cast<const Raw<T, E>*>(mine + (at * SOURCES + source) * 32 * BYTES);
    }
    __device__ __forceinline__ int ahead() const { return at + DEPTH >= SLOTS ? at + DEPTH - SLOTS : at + DEPTH; }
    __device__ __forceinline__ void next() { at = at + 1 == SLOTS ? 0 : at + 1; }
};

template <typename T, int E, int L, bool PAIRS, bool NORM>
__global__ void __launch_bounds__(WARPS * 32, FORWARD_A_SM) rotary_forward_kernel(const RotaryArgs a) {
    constexpr int HD = E * L, GROUPS = 32 / L;
    using R = Ring<T, E, AHEAD, 1>;
    __shared__ Shared share[WARPS];
    __shared__ __align__(16) float weights[2][HD];
    __shared__ __align__(16) char slots[WARPS][R::SLOTS * 32 * R::BYTES];
    const Place<E, L> me(a.rot);
    const int warp = threadIdx.x / 32, q_steps = (a.Hq + GROUPS - 1) / GROUPS, steps = q_steps + (a.Hk + GROUPS - 1) / GROUPS;
    R ring = {slots[warp] + me.lane * R::BYTES, 0};
    const int64_t stride = (int64_t)gridDim.x * WARPS;
    int64_t row = (int64_t)blockIdx.x * WARPS + warp, ahead = row;
    int step = 0;
    Source<T> from(a.q, a.q_stride, a.k, a.k_stride, row, me.at);
    auto fetch = [&](int slot) {
        if (ahead < a.N) {
            const bool key = step >= q_steps;
            const int h = (key ? step - q_steps : step) * GROUPS + me.group;
            if (h < (key ? a.Hk : a.Hq)) ring.copy(slot, 0, (key ? from.k : from.q) + h * HD);
            if (++step == steps) {
                step = 0;
                ahead += stride;
                from.next();
            }
        }
        cp_async_commit();
    };
    if (NORM) load_weights<T>(weights, a.q_gamma, a.k_gamma);
    Angles<E, PAIRS>::begin(share[warp]);
    __syncthreads();
#pragma unroll
    for (int d = 0; d < AHEAD; d++) fetch(d);
    int next = a.rot && row < a.N ? a.pos[row] : 0;
    for (; row < a.N; row += stride) {
        const int pos = next;
        if (a.rot && row + stride < a.N) next = a.pos[row + stride];
        Angles<E, PAIRS> ang;
        ang.of(pos, a.turns, me.at, a.rot, a.amplitude, share[warp]);
        auto heads = [&](int H, T* y, const float* weight) {
            float gamma[E];
            if (NORM) load_shared(gamma, weight + me.at);
            for (int h0 = 0; h0 < H; h0 += GROUPS) {
                const int h = h0 + me.group;
                cp_async_wait<AHEAD - 1>();
                float f[E];
                unpack(ring.read(0), f);
                fetch(ring.ahead());
                ring.next();
                if (NORM) {
                    times(f, rsqrtf(head_sum<L>(dot(f, f)) * (1.f / HD) + a.eps));
                    times(f, gamma);
                }
                rotate<E, PAIRS, false>(f, ang, me.other);
                if (h < H) store_e(y + h * HD, f);
            }
        };
        heads(a.Hq, (T*)a.qo + row * a.qo_stride + me.at, weights[0]);
        heads(a.Hk, (T*)a.ko + row * a.ko_stride + me.at, weights[1]);
    }
}

// With dn the gradient turned back and xhat = x rstd: dgamma = sum dn xhat,
// dx = rstd (dn gamma - xhat mean(dn gamma xhat)). A lane's values lie at the
// same place of every head it sees, so it keeps its share of dgamma in
// registers over all its rows; block sums go to partial [block][2][HD], which
// a column sum adds in a fixed order.
template <typename T, int E, int L, bool PAIRS, bool NORM>
__global__ void __launch_bounds__(WARPS * 32, BACKWARD_A_SM) rotary_backward_kernel(const RotaryArgs a,
                                                                               float* __restrict__ partial) {
    constexpr int HD = E * L, GROUPS = 32 / L, SOURCES = NORM ? 2 : 1;
    using R = Ring<T, E, AHEAD, SOURCES>;
    __shared__ Shared share[WARPS];
    __shared__ __align__(16) float weights[2][HD];
    __shared__ __align__(16) char slots[WARPS][R::SLOTS * SOURCES * 32 * R::BYTES];
    const Place<E, L> me(a.rot);
    const int warp = threadIdx.x / 32, q_steps = (a.Hq + GROUPS - 1) / GROUPS, steps = q_steps + (a.Hk + GROUPS - 1) / GROUPS;
    float aq[E], ak[E];
#pragma unroll
    for (int i = 0; i < E; i++) aq[i] = ak[i] = 0.f;
    R ring = {slots[warp] + me.lane * R::BYTES, 0};
    const int64_t stride = (int64_t)gridDim.x * WARPS;
    int64_t row = (int64_t)blockIdx.x * WARPS + warp, ahead = row;
    int step = 0;
    Source<T> dy(a.dqo, a.dqo_stride, a.dko, a.dko_stride, row, me.at), x(a.q, a.q_stride, a.k, a.k_stride, row, me.at);
    auto fetch = [&](int slot) {
        if (ahead < a.N) {
            const bool key = step >= q_steps;
            const int h = (key ? step - q_steps : step) * GROUPS + me.group;
            if (h < (key ? a.Hk : a.Hq)) {
                ring.copy(slot, 0, (key ? dy.k : dy.q) + h * HD);
                if (NORM) ring.copy(slot, SOURCES - 1, (key ? x.k : x.q) + h * HD);
            }
            if (++step == steps) {
                step = 0;
                ahead += stride;
                dy.next();
                x.next();
            }
        }
        cp_async_commit();
    };
    if (NORM) load_weights<T>(weights, a.q_gamma, a.k_gamma);
    Angles<E, PAIRS>::begin(share[warp]);
    __syncthreads();
#pragma unroll
    for (int d = 0; d < AHEAD; d++) fetch(d);
    int next = a.rot && row < a.N ? a.pos[row] : 0;
    for (; row < a.N; row += stride) {
        const int pos = next;
        if (a.rot && row + stride < a.N) next = a.pos[row + stride];
        Angles<E, PAIRS> ang;
        ang.of(pos, a.turns, me.at, a.rot, a.amplitude, share[warp]);
        auto heads = [&](int H, T* dx, const float* weight, float (&acc)[E]) {
            float gamma[E];
            if (NORM) load_shared(gamma, weight + me.at);
            for (int h0 = 0; h0 < H; h0 += GROUPS) {
                const int h = h0 + me.group;
                cp_async_wait<AHEAD - 1>();
                float d[E], v[E];
                unpack(ring.read(0), d);
                if (NORM) unpack(ring.read(SOURCES - 1), v);
                fetch(ring.ahead());
                ring.next();
                rotate<E, PAIRS, true>(d, ang, me.other);
                if (NORM) {
                    const float r = rsqrtf(head_sum<L>(dot(v, v)) * (1.f / HD) + a.eps);
                    times(v, r);
                    if (h < H) {
#pragma unroll
                        for (int i = 0; i < E; i += 2)
                            f2_unpack(f2_fma(f2_pack(d[i], d[i + 1]), f2_pack(v[i], v[i + 1]), f2_pack(acc[i], acc[i + 1])),
                                      acc[i], acc[i + 1]);
                    }
                    times(d, gamma);
                    const float in = head_sum<L>(dot(d, v)) * (-1.f / HD);
                    const uint64_t in2 = f2_pack(in, in), r2 = f2_pack(r, r);
#pragma unroll
                    for (int i = 0; i < E; i += 2)
                        f2_unpack(f2_mul(f2_fma(f2_pack(v[i], v[i + 1]), in2, f2_pack(d[i], d[i + 1])), r2), d[i], d[i + 1]);
                }
                if (h < H) store_e(dx + h * HD, d);
            }
        };
        heads(a.Hq, (T*)a.qo + row * a.qo_stride + me.at, weights[0], aq);
        heads(a.Hk, (T*)a.ko + row * a.ko_stride + me.at, weights[1], ak);
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
            if (me.group == 0) {
                sm[warp][0][me.at + i] = aq[i];
                sm[warp][1][me.at + i] = ak[i];
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * HD; c += WARPS * 32) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; w++) t += sm[w][c / HD][c % HD];
            partial[(int64_t)blockIdx.x * 2 * HD + c] = t;
        }
    }
}

// Blocks for N rows of one warp each, as many as stay resident.
int blocks_for(int N, int warps, int a_sm) {
    const int64_t rows = ((int64_t)N + warps - 1) / warps, most = (int64_t)gpt2_num_sms() * a_sm;
    return (int)(rows < most ? rows : most);
}
int forward_blocks(int N) { return blocks_for(N, WARPS, FORWARD_A_SM); }
int backward_blocks(int N) { return blocks_for(N, WARPS, BACKWARD_A_SM); }

template <typename T, int E, int L, bool PAIRS, bool NORM>
void start(const RotaryArgs& a, bool back, float* partial, cudaStream_t s) {
    if (back)
        rotary_backward_kernel<T, E, L, PAIRS, NORM><<<backward_blocks(a.N), WARPS * 32, 0, s>>>(a, partial);
    else rotary_forward_kernel<T, E, L, PAIRS, NORM><<<forward_blocks(a.N), WARPS * 32, 0, s>>>(a);
}

template <typename T, int E, int L> void start(const RotaryArgs& a, bool back, float* partial, cudaStream_t s) {
    if (a.interleaved) {
        if (a.norm) start<T, E, L, true, true>(a, back, partial, s);
        else start<T, E, L, true, false>(a, back, partial, s);
    } else {
        if (a.norm) start<T, E, L, false, true>(a, back, partial, s);
        else start<T, E, L, false, false>(a, back, partial, s);
    }
}

// E values a lane: rot (and in the half layout rot / 2) has to be a multiple of them.
template <typename T, int E> void start(const RotaryArgs& a, bool back, float* partial, cudaStream_t s) {
    switch (a.hd / E) {
        case 2: return start<T, E, 2>(a, back, partial, s);
        case 4: return start<T, E, 4>(a, back, partial, s);
        case 8: return start<T, E, 8>(a, back, partial, s);
        case 16: return start<T, E, 16>(a, back, partial, s);
        case 32: if constexpr (E == 4) return start<T, E, 32>(a, back, partial, s);
    }
}

}  // namespace

size_t rotary_backward_scratch(int N, int hd) { return (size_t)backward_blocks(N) * 2 * hd * 4; }

int launch_rotary(int dtype, const RotaryArgs& a, bool back, float* dq_gamma, float* dk_gamma, void* scratch,
                  cudaStream_t s) {
    float* partial = back && a.norm && (dq_gamma || dk_gamma) ? (float*)scratch : nullptr;
    if (dtype != GPT2_MODE_BF16) start<float, 4>(a, back, partial, s);
    else if (a.hd >= 16 && a.rot % (a.interleaved ? 8 : 16) == 0) start<bf16, 8>(a, back, partial, s);
    else start<bf16, 4>(a, back, partial, s);
    if (!partial) return 1;
    ColsumJob job = {partial, {dq_gamma, dk_gamma, nullptr}, backward_blocks(a.N), 2 * a.hd, a.hd, 0};
    return 1 + launch_colsum_jobs(&job, 1, s);
}
