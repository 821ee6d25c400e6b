// AdamW over many tensors in one launch, moments in 32 or in 8 bits
// (gpt2_op_adamw_many), and 8-bit moments read back (gpt2_op_adamw_many_states).
//
// The tensors' addresses travel as kernel parameters, so a call leaves nothing
// behind. A block serves CHUNK consecutive values of one tensor, found by a
// binary search over the tensors' first blocks; a thread holds four neighbours
// of each of its groups, a warp the 128 values that share an 8-bit moment's
// scale.
//
// 8-bit moments: m as e4m3 codes and v as e5m3 codes (no sign bit, bias 15)
// under a power of two for each 128 values, chosen so that the block's largest
// value lies in [2^7, 2^8) and [2^14, 2^15): 17 and 31 binades below it can be
// told apart. A power of two keeps codes that did not change exact from step to
// step, and one byte holds it. Rounding goes up or down by 16 random bits, so
// that the stored moment is right on average: with three mantissa bits,
// rounding to nearest would never let v shrink at beta2 = 0.95 or above (a step
// changes it by 5% at most, half a code is 6%). A v above 0 keeps at least the
// lowest code, so that no m meets a v that was rounded away. The parameter's
// own update uses m and v before they are rounded.
//
// HBM bounds it: per parameter 8 bytes of master, 2 of its bf16 copy, the
// gradient, and 16 or 4 + 1/32 of moments.
#include "common.cuh"
#include "launch.h"

#include <cuda_fp16.h>
#include <math.h>

namespace {

constexpr int THREADS = 256;
constexpr int GROUPS = 2;                       // groups of four values a thread
constexpr int CHUNK = THREADS * 4 * GROUPS;     // values a block of the update
constexpr int WIDE = 8192;                      // and of the passes that only read or only decode
constexpr int SCALE_BLOCK = 128;                // values that share a scale: a warp's group

struct Entry {
    float* master;
    bf16* param;
    const void* grad;
    void *m, *v;
    uint8_t *m_scale, *v_scale;
    int64_t n;
    float decay;
    int first, first_wide;  // first block of this tensor, in chunks and in wide ones
    int aligned;            // every address allows four values at once
};

// MOST tensors a launch: few fit the classic 4 KB of parameters, whose upload is cheaper.
template <int MOST> struct Batch {
    Entry e[MOST];
    int n, base;  // base: the first tensor's number in the call
};
constexpr int FEW = 48, MANY = 380;
static_assert(sizeof(Batch<FEW>) <= 4000 && sizeof(Batch<MANY>) <= 32000, "kernel parameters");

struct Values {
    float lr, b1, b2, eps, inv_bc1, inv_bc2, grad_scale, max_norm;
    const float* norm;  // or null
    uint64_t key;
};

template <int Entry::*FIRST, int MOST> __device__ __forceinline__ int find(const Batch<MOST>& b, int block) {
    int lo = 0, hi = b.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.e[mid].*FIRST <= block) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ uint64_t mix(uint64_t z) {  // the finaliser of splitmix64
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ULL;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBULL;
    return z ^ (z >> 31);
}

// (Without the hint that the values are read once.)
__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
}
__device__ __forceinline__ void load4(const bf16* p, float (&f)[4]) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    f[0] = __uint_as_float(u.x << 16); f[1] = __uint_as_float(u.x & 0xFFFF0000u);
    f[2] = __uint_as_float(u.y << 16); f[3] = __uint_as_float(u.y & 0xFFFF0000u);
}

constexpr uint64_t GOLDEN = 0x9E3779B97F4A7C15ULL;

// Four neighbours of n values from i on; what lies behind the end reads as 0 and is not written.
__device__ __forceinline__ void get4(const float* p, int64_t i, int64_t n, bool whole, float (&f)[4]) {
    if (whole) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(p + i));
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++) f[j] = i + j < n ? p[i + j] : 0.f;
    }
}
__device__ __forceinline__ void get4(const bf16* p, int64_t i, int64_t n, bool whole, float (&f)[4]) {
    if (whole) {
        const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p + i));
        f[0] = __uint_as_float(u.x << 16); f[1] = __uint_as_float(u.x & 0xFFFF0000u);
        f[2] = __uint_as_float(u.y << 16); f[3] = __uint_as_float(u.y & 0xFFFF0000u);
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++) f[j] = i + j < n ? __bfloat162float(p[i + j]) : 0.f;
    }
}
__device__ __forceinline__ uint32_t get4(const uint8_t* p, int64_t i, int64_t n, bool whole) {
    if (whole) return __ldcs(reinterpret_cast<const uint32_t*>(p + i));
    uint32_t u = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) u |= i + j < n ? (uint32_t)p[i + j] << (8 * j) : 0u;
    return u;
}
__device__ __forceinline__ void put4(float* p, int64_t i, int64_t n, bool whole, const float (&f)[4]) {
    if (whole) {
        __stcs(reinterpret_cast<float4*>(p + i), make_float4(f[0], f[1], f[2], f[3]));
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (i + j < n) p[i + j] = f[j];
    }
}
__device__ __forceinline__ void put4(bf16* p, int64_t i, int64_t n, bool whole, const float (&f)[4]) {
    if (whole) {
        uint2 u;
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
        h[0] = __floats2bfloat162_rn(f[0], f[1]);
        h[1] = __floats2bfloat162_rn(f[2], f[3]);
        *reinterpret_cast<uint2*>(p + i) = u;
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (i + j < n) p[i + j] = __float2bfloat16_rn(f[j]);
    }
}
__device__ __forceinline__ void put4(uint8_t* p, int64_t i, int64_t n, bool whole, uint32_t u) {
    if (whole) {
        __stcs(reinterpret_cast<uint32_t*>(p + i), u);
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (i + j < n) p[i + j] = (uint8_t)(u >> (8 * j));
    }
}

// Four codes (a word) as fp32, without their scale. m: two e4m3 codes a conversion. v: a code is the top byte of an
// fp16 number without its sign bit.
__device__ __forceinline__ void decode_m(uint32_t w, float (&f)[4]) {
#pragma unroll
    for (int p = 0; p < 2; p++) {
        uint32_t h;
        asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(h) : "r"(w >> (16 * p)));
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
        f[2 * p] = x.x;
        f[2 * p + 1] = x.y;
    }
}
__device__ __forceinline__ void decode_v(uint32_t w, float (&f)[4]) {
#pragma unroll
    for (int p = 0; p < 2; p++) {
        const uint32_t h = __byte_perm(w, 0, p ? 0x4342 : 0x4140) << 7;
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
        f[2 * p] = x.x;
        f[2 * p + 1] = x.y;
    }
}
__device__ __forceinline__ float scale_of(uint8_t b) { return __uint_as_float((b < 1 ? 1u : b > 254 ? 254u : b) << 23); }

// The code of y >= 0 in the top byte, given y under its scale, times 2^(bias - 127): bits 20 to 27 of the fp32 number
// are the code, an fp32 subnormal holding what is below the code's lowest whole exponent. Adding 16 random bits right
// below the code's last one carries into it with the probability (what is left over the lower code) / (the codes'
// distance). One product (bits x 16 + random bits x 256) shifts both to the top: the integer pipe has half the rate of
// the FMA pipe, and it bounds the kernel. random: the 16 bits in the middle two bytes.
__device__ __forceinline__ uint32_t encode(float y, uint32_t random) { return __float_as_uint(y) * 16u + random; }
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// The scale byte of a block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t largest, int top) {
    const int b = (int)(largest >> 23) - top;
    return b < 1 ? 1u : (uint32_t)b;
}
// The square root and the quotient of 8-bit moments' updates are the hardware's (2^-22 of a step, where a stored
// moment is off by up to 2^-4): the IEEE forms cost a third of the kernel.
template <bool EIGHT> __device__ __forceinline__ float step_of(float m, float v, float eps) {
    if (!EIGHT) return m / (sqrtf(v) + eps);
    float root;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(root) : "f"(v));
    return __fdividef(m, root + eps);
}

// A block's chunk of a tensor: all loads of the thread's groups first, then one group after another (what is stored
// may be what a later group loads, as far as the compiler knows: it moves no load over a store). WHOLE: the chunk lies
// inside the tensor and every address allows four values at once.
template <typename G, bool EIGHT, bool WHOLE>
__device__ __forceinline__ void adamw_chunk(const Entry& e, const Values& h, int64_t base, uint64_t draw) {
    const int64_t n = e.n;
    float gs = h.grad_scale;
    if (h.norm) gs *= fminf(1.f, h.max_norm / __fadd_rn(__fmul_rn(*h.norm, fabsf(h.grad_scale)), 1e-6f));
    float th[GROUPS][4], g[GROUPS][4], m[GROUPS][4], v[GROUPS][4];
    uint32_t cm[GROUPS], cv[GROUPS];
    uint8_t bm[GROUPS], bv[GROUPS];
    auto whole = [&](int u) { return WHOLE || (e.aligned && base + u * (THREADS * 4) + 4 <= n); };
#pragma unroll
    for (int u = 0; u < GROUPS; u++) {
        const int64_t i = base + u * (THREADS * 4);
        get4(e.master, i, n, whole(u), th[u]);
        get4((const G*)e.grad, i, n, whole(u), g[u]);
        if (EIGHT) {
            const bool in = WHOLE || i < n;
            bm[u] = in ? e.m_scale[i / SCALE_BLOCK] : 0;
            bv[u] = in ? e.v_scale[i / SCALE_BLOCK] : 0;
            cm[u] = get4((const uint8_t*)e.m, i, n, whole(u));
            cv[u] = get4((const uint8_t*)e.v, i, n, whole(u));
        } else {
            get4((const float*)e.m, i, n, whole(u), m[u]);
            get4((const float*)e.v, i, n, whole(u), v[u]);
        }
    }
    const float b1c = 1.f - h.b1, b2c = 1.f - h.b2;
#pragma unroll
    for (int u = 0; u < GROUPS; u++) {
        const int64_t i = base + u * (THREADS * 4);
        if (!WHOLE && i - (threadIdx.x & 31) * 4 >= n) break;  // the whole warp
        if (EIGHT) {
            const float ms = scale_of(bm[u]), vs = scale_of(bv[u]);
            decode_m(cm[u], m[u]);
            decode_v(cv[u], v[u]);
#pragma unroll
            for (int j = 0; j < 4; j++) m[u][j] *= ms, v[u][j] *= vs;
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float gj = g[u][j] * gs;
            if (EIGHT) {  // (each product and sum rounded on its own: the codes that follow are everyone's)
                m[u][j] = __fadd_rn(__fmul_rn(h.b1, m[u][j]), __fmul_rn(b1c, gj));
                v[u][j] = __fadd_rn(__fmul_rn(h.b2, v[u][j]), __fmul_rn(b2c, __fmul_rn(gj, gj)));
            } else {
                m[u][j] = h.b1 * m[u][j] + b1c * gj;
                v[u][j] = h.b2 * v[u][j] + b2c * gj * gj;
            }
            th[u][j] -= h.lr * (step_of<EIGHT>(m[u][j] * h.inv_bc1, v[u][j] * h.inv_bc2, h.eps) + e.decay * th[u][j]);
        }
        put4(e.master, i, n, whole(u), th[u]);
        if (e.param) put4(e.param, i, n, whole(u), th[u]);
        if (EIGHT) {
            float fm = 0.f, fv = 0.f, check = 0.f;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                fm = fmaxf(fm, fabsf(m[u][j]));
                fv = fmaxf(fv, fabsf(v[u][j]));
                check = fmaf(m[u][j], 0.f, fmaf(v[u][j], 0.f, check));  // 0, or NaN where one is not finite
            }
            const bool odd = __any_sync(0xffffffffu, check != 0.f);
            if (odd) {  // what is not finite leaves the scale alone
                fm = fv = 0.f;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    if (isfinite(m[u][j])) fm = fmaxf(fm, fabsf(m[u][j]));
                    if (isfinite(v[u][j])) fv = fmaxf(fv, fabsf(v[u][j]));
                }
            }
            const uint32_t am = scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(fm)), 7);
            const uint32_t av = scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(fv)), 14);
            const float im = __uint_as_float((254u - am) << 23), iv = __uint_as_float((254u - av) << 23);
            uint32_t x[4], y[4];
#pragma unroll
            for (int p = 0; p < 2; p++) {
                const uint64_t r = mix(draw + p * GOLDEN);
#pragma unroll
                for (int o = 0; o < 2; o++) {
                    const int j = 2 * p + o;
                    const uint32_t w = (uint32_t)(r >> (32 * o));
                    x[j] = encode(fabsf(m[u][j]) * im * 0x1p-120f, __byte_perm(w, 0, 0x4104));
                    // (0x1p-129f, a subnormal, is the lowest code)
                    const float least = fminf(v[u][j] * 0x1p120f, 0x1p-129f);
                    y[j] = encode(fmaxf(v[u][j] * iv * 0x1p-112f, least), __byte_perm(w, 0, 0x4324));
                    if (odd) {
                        if (!isfinite(m[u][j])) x[j] = 0x7F000000u;
                        if (!isfinite(v[u][j])) y[j] = 0xFF000000u;
                    }
                }
            }
            const uint32_t sign = top_bytes(__float_as_uint(m[u][0]), __float_as_uint(m[u][1]), __float_as_uint(m[u][2]),
                                            __float_as_uint(m[u][3]));
            const uint32_t wm = top_bytes(x[0], x[1], x[2], x[3]) | (sign & 0x80808080u);
            const uint32_t wv = top_bytes(y[0], y[1], y[2], y[3]);
            draw += (uint64_t)(THREADS * 2) * GOLDEN;
            put4((uint8_t*)e.m, i, n, whole(u), wm);
            put4((uint8_t*)e.v, i, n, whole(u), wv);
            if ((threadIdx.x & 31) == 0) {
                e.m_scale[i / SCALE_BLOCK] = (uint8_t)am;
                e.v_scale[i / SCALE_BLOCK] = (uint8_t)av;
            }
        } else {
            put4((float*)e.m, i, n, whole(u), m[u]);
            put4((float*)e.v, i, n, whole(u), v[u]);
        }
    }
}

template <int MOST, typename G, bool EIGHT>
__global__ void __launch_bounds__(THREADS) adamw_many_kernel(const __grid_constant__ Batch<MOST> b, const Values h) {
    // from the end: the norm's pass has just read the last gradients, which L2 still holds
    const int block = gridDim.x - 1 - blockIdx.x;
    const int k = find<&Entry::first>(b, block);
    const Entry& e = b.e[k];
    const int64_t first = (int64_t)(block - e.first) * CHUNK, base = first + threadIdx.x * 4;
    const uint64_t draw = h.key + (((uint64_t)(b.base + k) << 40) + (uint64_t)base / 2) * GOLDEN;
    if (e.aligned && first + CHUNK <= e.n) adamw_chunk<G, EIGHT, true>(e, h, base, draw);
    else adamw_chunk<G, EIGHT, false>(e, h, base, draw);
}

// A sum of squares in two fp32 numbers: four squares at a time, and what a rounding of `sum` drops goes to `rest`. The
// norm scales every gradient, and a last bit of it can move codes of 8-bit moments: so it is summed to about its last
// bit, the four squares' roundings being of either sign and far below the whole. (124M values: 81 us; each square exact
// and on its own 100, in plain fp32 sums 80; in 64 bits the pass would take twice the time of its reads.)
struct Squares {
    float sum = 0.f, rest = 0.f;
    __device__ __forceinline__ void add(const float (&g)[4]) {
        const float p = fmaf(g[3], g[3], fmaf(g[2], g[2], fmaf(g[1], g[1], g[0] * g[0])));
        const float t = __fadd_rn(sum, p), z = __fsub_rn(t, sum);
        rest = __fadd_rn(rest, __fadd_rn(__fsub_rn(sum, __fsub_rn(t, z)), __fsub_rn(p, z)));
        sum = t;
    }
};

// Sums of squares of the gradients: a block takes every gridDim.x-th chunk and adds in a fixed order.
template <int MOST, typename G>
__global__ void __launch_bounds__(THREADS) sumsq_many_kernel(const __grid_constant__ Batch<MOST> b, int chunks,
                                                             double* __restrict__ partial) {
    __shared__ double sh[THREADS / 32];
    Squares acc[2];
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Entry& e = b.e[find<&Entry::first_wide>(b, c)];
        const int64_t n = e.n, first = (int64_t)(c - e.first_wide) * WIDE, base = first + threadIdx.x * 4;
        constexpr int LOADS = WIDE / (THREADS * 4);
        if (e.aligned && first + WIDE <= n) {
            float g[LOADS][4];
#pragma unroll
            for (int u = 0; u < LOADS; u++) load4((const G*)e.grad + base + u * (THREADS * 4), g[u]);
#pragma unroll
            for (int u = 0; u < LOADS; u++) acc[u % 2].add(g[u]);
        } else {
#pragma unroll 4
            for (int u = 0; u < LOADS; u++) {
                const int64_t i = base + u * (THREADS * 4);
                if (i >= n) break;
                float g[4];
                get4((const G*)e.grad, i, n, e.aligned && i + 4 <= n, g);
                acc[u % 2].add(g);
            }
        }
    }
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < 2; j++)  // (a sum past fp32's range is infinite and what it dropped is NaN)
        s += (double)acc[j].sum + (isinf(acc[j].sum) ? 0.0 : (double)acc[j].rest);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; w++) t += sh[w];
        partial[blockIdx.x] = t;
    }
}

__global__ void __launch_bounds__(1024) norm_many_kernel(float* __restrict__ norm, float* __restrict__ out,
                                                         const double* __restrict__ partial, int n) {
    __shared__ double sh[32];
    double v = 0.0;
    for (int i = threadIdx.x; i < n; i += 1024) v += partial[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int w = 0; w < 32; w++) t += sh[w];
        *norm = (float)sqrt(t);
        if (out) *out = *norm;
    }
}

// Eight codes a thread and load, all loads of a chunk first. The values' places travel in master and param.
template <int MOST, typename T>
__global__ void __launch_bounds__(THREADS) states_many_kernel(const __grid_constant__ Batch<MOST> b) {
    const Entry& e = b.e[find<&Entry::first_wide>(b, blockIdx.x)];
    const int64_t n = e.n, first = (int64_t)((int)blockIdx.x - e.first_wide) * WIDE;
    const uint8_t *m = (const uint8_t*)e.m, *v = (const uint8_t*)e.v;
    T *mo = (T*)(void*)e.master, *vo = (T*)(void*)e.param;
    if (!e.aligned || first + WIDE > n) {
        for (int64_t i = first + threadIdx.x * 4; i < min(n, first + WIDE); i += THREADS * 4) {
            const bool whole = e.aligned && i + 4 <= n;
            const float ms = scale_of(e.m_scale[i / SCALE_BLOCK]), vs = scale_of(e.v_scale[i / SCALE_BLOCK]);
            float x[4], y[4];
            decode_m(get4(m, i, n, whole), x);
            decode_v(get4(v, i, n, whole), y);
#pragma unroll
            for (int j = 0; j < 4; j++) x[j] *= ms, y[j] *= vs;
            put4(mo, i, n, whole, x);
            put4(vo, i, n, whole, y);
        }
        return;
    }
    constexpr int LOADS = WIDE / (THREADS * 8);
    uint2 cm[LOADS], cv[LOADS];
    float sm[LOADS], sv[LOADS];
#pragma unroll
    for (int u = 0; u < LOADS; u++) {
        const int64_t i = first + (u * THREADS + threadIdx.x) * 8;
        cm[u] = __ldcs(reinterpret_cast<const uint2*>(m + i));
        cv[u] = __ldcs(reinterpret_cast<const uint2*>(v + i));
        sm[u] = scale_of(e.m_scale[i / SCALE_BLOCK]);
        sv[u] = scale_of(e.v_scale[i / SCALE_BLOCK]);
    }
#pragma unroll
    for (int u = 0; u < LOADS; u++) {
        const int64_t i = first + (u * THREADS + threadIdx.x) * 8;
        float f[8];
        auto decoded = [&](auto decode, uint2 c, float s, T* to) {
            decode(c.x, reinterpret_cast<float(&)[4]>(f[0]));
            decode(c.y, reinterpret_cast<float(&)[4]>(f[4]));
#pragma unroll
            for (int j = 0; j < 8; j++) f[j] *= s;
            store8(to + i, f);
        };
        decoded([](uint32_t w, float (&x)[4]) { decode_m(w, x); }, cm[u], sm[u], mo);
        decoded([](uint32_t w, float (&x)[4]) { decode_v(w, x); }, cv[u], sv[u], vo);
    }
}

bool at16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// The entries of tensors [i0, i1) and the blocks that they take, in chunks and in wide ones.
template <int MOST, typename Fill>
void gather(Batch<MOST>& b, const gpt2_adamw_tensor* t, int i0, int i1, Fill fill, int& blocks, int& wide) {
    blocks = wide = 0;
    b.n = 0;
    b.base = i0;
    for (int i = i0; i < i1; i++) {
        Entry& e = b.e[b.n++];
        e = {t[i].master, (bf16*)t[i].param_bf16, t[i].grad, t[i].m, t[i].v, t[i].m_scale, t[i].v_scale, t[i].n,
             t[i].weight_decay, blocks, wide, 0};
        fill(e, i);
        e.aligned = at16(e.master) && at16(e.param) && at16(e.grad) && at16(e.m) && at16(e.v);
        blocks += (int)((e.n + CHUNK - 1) / CHUNK);
        wide += (int)((e.n + WIDE - 1) / WIDE);
    }
}

// Calls go(batch, blocks, wide blocks) for the tensors in as few launches as they fit.
template <typename Fill, typename Go> int in_batches(const gpt2_adamw_tensor* t, int n, Fill fill, Go go) {
    int launches = 0, blocks, wide;
    for (int i = 0; i < n;) {
        const int left = n - i;
        if (left <= FEW) {
            Batch<FEW> b;
            gather(b, t, i, n, fill, blocks, wide);
            if (blocks) launches++, go(b, blocks, wide);
            i = n;
        } else {
            const int to = left < MANY ? n : i + MANY;
            Batch<MANY> b;
            gather(b, t, i, to, fill, blocks, wide);
            if (blocks) launches++, go(b, blocks, wide);
            i = to;
        }
    }
    return launches;
}

template <int MOST, typename G>
void start_adamw(const Batch<MOST>& b, int blocks, int bits, const Values& h, cudaStream_t s) {
    if (bits == 8) adamw_many_kernel<MOST, G, true><<<blocks, THREADS, 0, s>>>(b, h);
    else adamw_many_kernel<MOST, G, false><<<blocks, THREADS, 0, s>>>(b, h);
}

int sumsq_blocks() { return gpt2_num_sms() * 8; }

uint64_t host_mix(uint64_t z) {
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ULL;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBULL;
    return z ^ (z >> 31);
}

}  // namespace

// The norm, then a partial sum for each block.
size_t adamw_many_scratch(const gpt2_adamw_tensor* t, int n) {
    int64_t wide = 0;
    for (int i = 0; i < n; i++) wide += (t[i].n + WIDE - 1) / WIDE;
    const int64_t most = (int64_t)sumsq_blocks() * (n / MANY + 1);
    return 256 + (size_t)(wide < most ? wide : most) * 8;
}

int launch_adamw_many(const gpt2_adamw_tensor* t, int n, int grad_dtype, int bits, float lr, float b1, float b2,
                      float eps, float grad_scale, float max_norm, float* grad_norm, int step, uint64_t seed,
                      void* scratch, cudaStream_t s) {
    const double bc1 = 1.0 - pow((double)b1, (double)step), bc2 = 1.0 - pow((double)b2, (double)step);
    Values h = {lr, b1, b2, eps, (float)(1.0 / bc1), (float)(1.0 / bc2), grad_scale, max_norm, nullptr,
                host_mix(seed + (uint64_t)step * 0x9E3779B97F4A7C15ULL)};
    int launches = 0;
    auto as_is = [](Entry&, int) {};
    if (max_norm > 0.f || grad_norm) {
        float* norm = (float*)scratch;
        double* partial = (double*)(norm + 64);
        int at = 0;
        launches += in_batches(t, n, as_is, [&](const auto& b, int, int wide) {
            constexpr int MOST = sizeof(b.e) / sizeof(Entry);
            const int grid = wide < sumsq_blocks() ? wide : sumsq_blocks();
            if (grad_dtype == GPT2_MODE_BF16)
                sumsq_many_kernel<MOST, bf16><<<grid, THREADS, 0, s>>>(b, wide, partial + at);
            else
                sumsq_many_kernel<MOST, float><<<grid, THREADS, 0, s>>>(b, wide, partial + at);
            at += grid;
        });
        norm_many_kernel<<<1, 1024, 0, s>>>(norm, grad_norm, partial, at);
        launches++;
        if (max_norm > 0.f) h.norm = norm;
    }
    return launches + in_batches(t, n, as_is, [&](const auto& b, int blocks, int) {
        constexpr int MOST = sizeof(b.e) / sizeof(Entry);
        if (grad_dtype == GPT2_MODE_BF16) start_adamw<MOST, bf16>(b, blocks, bits, h, s);
        else start_adamw<MOST, float>(b, blocks, bits, h, s);
    });
}

int launch_adamw_many_states(const gpt2_adamw_tensor* t, void* const* m_values, void* const* v_values, int n,
                             int dtype, cudaStream_t s) {
    auto places = [&](Entry& e, int i) {
        e.master = (float*)m_values[i];
        e.param = (bf16*)v_values[i];
        e.grad = nullptr;
    };
    return in_batches(t, n, places, [&](const auto& b, int, int wide) {
        constexpr int MOST = sizeof(b.e) / sizeof(Entry);
        if (dtype == GPT2_MODE_BF16) states_many_kernel<MOST, bf16><<<wide, THREADS, 0, s>>>(b);
        else states_many_kernel<MOST, float><<<wide, THREADS, 0, s>>>(b);
    });
}
