// Log-probabilities of given tokens, with entropy and the top alternatives,
// and their gradient. Both are bound by HBM: the logits are read once (and
// the gradient written once); everything else stays in registers. 32768 rows of
// 50257 bf16 logits take 498 us (6.6 TB/s), the gradient of 8192 242 us (6.8).
//
// With m the row's maximum, d_j = (z_j - m) log2(e) and e_j = 2^d_j,
//   S = sum e_j, T = sum e_j d_j:  lse = m + ln S,  entropy = ln S - ln2 T / S,
//   log p_j = (z_j - m) - ln S (not z_j - lse: lse carries a rounding of its own
//   size, which far from 0 is more than a sure token's log-probability),
// in one pass: a thread keeps its own m, S, T and moves them to a new maximum
// by S' = f S, T' = f (T + S (m - m') log2(e)), f = 2^((m - m') log2(e)).
#include "common.cuh"
#include "launch.h"
#include "tc_common.cuh"

#include <cooperative_groups.h>

namespace {

namespace cg = cooperative_groups;
using namespace tc;

constexpr int BATCH = 4;      // 16-byte vectors a thread has in flight
constexpr int MAX_SPLIT = 8;  // blocks (a cluster) that share a row
constexpr int TOP_SPLIT = 4;  // with alternatives: joining eight lists takes longer than eight save
constexpr int MAX_K = 64;
constexpr int CAND = 512;     // candidates for the top k that fit in shared memory
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

template <typename T> constexpr int VEC = 16 / sizeof(T);  // values of a 16-byte vector

__device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void pack(uint4& u, const float (&f)[8]) {
    uint32_t* w = &u.x;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
}
__device__ __forceinline__ void pack(uint4& u, const float (&f)[4]) {
    u = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

// Maxima that a NaN passes through.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// A logit's place in the order (larger logits larger, -0 as 0, NaN largest)
// above its column's (lower columns larger): unique within a row, neither 0 nor ~0.
__device__ __forceinline__ uint64_t order_key(float z, int col) {
    const int b = z != z ? 0x7FFFFFFE : __float_as_int(z + 0.f);
    const uint32_t u = (uint32_t)(b < 0 ? ~b : b ^ 0x80000000);
    return ((uint64_t)u << 32) | (uint32_t)~col;
}
__device__ __forceinline__ int key_col(uint64_t k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ float key_logit(uint64_t k) {
    const uint32_t u = (uint32_t)(k >> 32);
    return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// Maximum, sum and weighted sum of some of a row's values.
struct Stats {
    float m, s, t;
};
// The reference that d is taken against: 0 before any finite value, so that
// e = 2^-inf = 0 and nothing becomes inf - inf.
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ void move_to(Stats& x, float m) {
    if (x.m == m) return;
    if (x.m == -INFINITY) {
        x.m = m;  // s = t = 0
        return;
    }
    const float d = (x.m - m) * LOG2E, f = ex2_approx(d);
    x.t = f == 0.f ? 0.f : f * (x.t + x.s * d);
    x.s *= f;
    x.m = m;
}
// The same for all of LANES neighbouring lanes: the maximum first, then each
// lane's sums moved to it once and added (x + y and y + x: the same bits in
// every lane).
template <int LANES> __device__ __forceinline__ Stats join(Stats x) {
    float m = x.m;
#pragma unroll
    for (int o = LANES / 2; o > 0; o /= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    move_to(x, m);
#pragma unroll
    for (int o = LANES / 2; o > 0; o /= 2) {
        x.s += __shfl_xor_sync(0xffffffffu, x.s, o);
        x.t += __shfl_xor_sync(0xffffffffu, x.t, o);
    }
    return x;
}

// N values into x, whose maximum is already at least theirs, 2^d taken
//   fast: with d = z log2(e) - m log2(e) in one step. The rounding of m log2(e)
//     shifts every d alike, by delta (below 2^-11 while |m| is moderate), which
//     is taken out of the sums: S 2^-delta, 2^-delta (T - delta S) (left in, the
//     largest weight is not 1 and log-probabilities are off by |m| 2^-24; 495 us
//     for the 32768 rows then, 498 so; m log2(e) rounded to a whole number, whose
//     shift goes out once a row: 506). e d is a NaN where z is -inf, which the
//     caller sees in x.t;
//   else: from the difference z - m, exact for the largest, and with d bounded
//     (e is 0 below -150, and 0 * -inf must not count): for masks from -1e38 to
//     -inf and far-off rows.
template <bool FAST, int N> __device__ __forceinline__ void add_values(const float (&f)[N], Stats& x) {
    const float m = reference(x.m), ml = -m * LOG2E;
    const uint64_t m2 = FAST ? f2_pack(ml, ml) : f2_pack(m, m), l2e = f2_pack(LOG2E, LOG2E);
    uint64_t s2[2] = {0, 0}, t2[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        const uint64_t z2 = f2_pack(f[j], f[j + 1]);
        uint64_t d2 = FAST ? f2_fma(z2, l2e, m2) : f2_mul(f2_sub(z2, m2), l2e);
        float d0, d1;
        f2_unpack(d2, d0, d1);
        const uint64_t e2 = f2_pack(ex2_approx(d0), ex2_approx(d1));
        if (!FAST) d2 = f2_pack(fmaxf(d0, -200.f), fmaxf(d1, -200.f));
        s2[(j >> 1) & 1] = f2_add(s2[(j >> 1) & 1], e2);
        t2[(j >> 1) & 1] = f2_fma(e2, d2, t2[(j >> 1) & 1]);
    }
    float a, b;
    f2_unpack(f2_add(s2[0], s2[1]), a, b);
    float s = a + b;
    f2_unpack(f2_add(t2[0], t2[1]), a, b);
    float t = a + b;
    if (FAST) {
        const float delta = fmaf(m, LOG2E, ml), y = -LN2 * delta, c = fmaf(y, fmaf(y, 0.5f, 1.f), 1.f);  // 2^-delta
        t = c * fmaf(-delta, s, t);
        s *= c;
    }
    x.s += s;
    x.t += t;
}
template <int N> __device__ __forceinline__ void raise(const float (&f)[N], Stats& x) {
    float m[2] = {x.m, -INFINITY};
#pragma unroll
    for (int j = 0; j < N; j += 2) m[(j >> 1) & 1] = max_nan(m[(j >> 1) & 1], f[j], f[j + 1]);
    const float top = max_nan(m[0], m[1]);
    if (!(top <= x.m)) move_to(x, top);
}

// What a row's sums say.
struct Row {
    float m, ln_s;  // ln S: at least 0 but for rounding, as the largest logit's own weight is 1 (0 for m = +-inf)
    __device__ __forceinline__ Row(float m, float ln_s) : m(m), ln_s(ln_s) {}
    __device__ __forceinline__ explicit Row(const Stats& x)
        : m(x.m), ln_s(isinf(x.m) ? 0.f : max_nan(LN2 * log2f(x.s), 0.f)) {}
    __device__ __forceinline__ float lse() const { return m + ln_s; }
    __device__ __forceinline__ float entropy(const Stats& x) const {
        return m == -INFINITY ? 0.f : max_nan(ln_s - LN2 * (x.t / x.s), 0.f);
    }
    __device__ __forceinline__ float logp(float z) const { return m == -INFINITY ? -INFINITY : (z - m) - ln_s; }
};

// The split-th part of a row's vectors: [first, last).
__device__ __forceinline__ void part(int nv, int split, int rank, int& first, int& last) {
    const int per = (nv + split - 1) / split;
    first = min(rank * per, nv);
    last = min(first + per, nv);
}

// Whole vectors into x.
template <typename T, int N> __device__ __forceinline__ void add_batch(const uint4 (&u)[N], Stats& x) {
    float f[N * VEC<T>];
#pragma unroll
    for (int b = 0; b < N; b++) {
        float g[VEC<T>];
        unpack(u[b], g);
#pragma unroll
        for (int j = 0; j < VEC<T>; j++) f[b * VEC<T> + j] = g[j];
    }
    raise(f, x);
    const Stats was = x;
    const bool near = fabsf(x.m) < 1e4f;
    if (near) add_values<true>(f, x);
    if (!near || x.t != x.t) {
        x = was;
        add_values<false>(f, x);
    }
}
// Vector v, which V may cut.
template <typename T> __device__ __forceinline__ void add_vector(const uint4& u, int v, int V, Stats& x) {
    float f[VEC<T>];
    unpack(u, f);
#pragma unroll
    for (int j = 0; j < VEC<T>; j++)
        if (v * VEC<T> + j >= V) f[j] = -INFINITY;
    raise(f, x);
    add_values<false>(f, x);
}

// The first columns of vectors [v0, v1) whose logits are at the bound itself, by a warp: behind the n places of
// out that are taken, up to k. Returns the places taken then.
template <typename T>
__device__ __forceinline__ int add_equal(const uint4* zv, int v0, int v1, int V, uint32_t bound, int n, int k,
                                         uint64_t* out) {
    const int lane = threadIdx.x & 31;
    for (; n < k && v0 < v1; v0 += 32) {
        const int v = v0 + lane;
        uint64_t q[VEC<T>];
        float g[VEC<T>];
        unpack(v < v1 ? __ldg(zv + v) : make_uint4(0, 0, 0, 0), g);
        int own = 0;
#pragma unroll
        for (int j = 0; j < VEC<T>; j++) {
            q[j] = order_key(g[j], v * VEC<T> + j);
            if ((uint32_t)(q[j] >> 32) != bound || v >= v1 || v * VEC<T> + j >= V) q[j] = 0;
            own += q[j] != 0;
        }
        int to = own;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, to, o);
            if (lane >= o) to += y;
        }
        const int all = __shfl_sync(0xffffffffu, to, 31);
        to += n - own;
#pragma unroll
        for (int j = 0; j < VEC<T>; j++)
            if (q[j]) {
                if (to < k) out[to] = q[j];
                to++;
            }
        n += all;
    }
    return min(n, k);
}

// A row is read by `split` blocks (a cluster), thread t of NT taking every
// NT-th vector of the block's part. Top k: each thread knows its
// largest logit, which gives a lower bound of the block's k-th largest; the few
// threads that reach it have their vectors looked through again (from L2) for
// what reaches the bound: some more than k candidates, ranked by counting. More
// than CAND are equal logits at the bound, as in a row with fewer than k tokens
// left unmasked: those above it are found in the same way, then the first
// columns at it (4096 rows with all but 5 masked: 95 us; taken one by one
// 1670). Only where CAND are above it (a row that rises, its largest logits all
// in a few threads) are they taken one by one. The blocks' lists and sums meet
// in the first block's shared memory.
template <typename T, int NT, bool TOP>
__global__ void __launch_bounds__(NT)
    logprobs_kernel(float* __restrict__ logp, float* __restrict__ lse, float* __restrict__ entropy,
                    float* __restrict__ top_logp, int32_t* __restrict__ top_ids, int k, const T* __restrict__ logits,
                    const int32_t* __restrict__ targets, int V, int Vp, int split, int* status) {
    __shared__ Stats ws[NT / 32], cs[MAX_SPLIT];
    __shared__ uint64_t keys[TOP ? CAND : 1], lists[TOP ? TOP_SPLIT * MAX_K : 1];
    __shared__ __align__(16) uint32_t maxima[TOP ? NT : 4];
    __shared__ uint32_t bound;
    __shared__ int count;
    __shared__ float whole[2];  // the row's maximum and ln S
    const int row = blockIdx.x / split, rank = blockIdx.x - row * split;
    const int tid = threadIdx.x, lane = tid & 31;
    const T* z = logits + (int64_t)row * Vp;
    const uint4* zv = reinterpret_cast<const uint4*>(z);
    const int nv = (V + VEC<T> - 1) / VEC<T>;
    int v0, v1;
    part(nv, split, rank, v0, v1);
    // every block of the cluster is running before another writes to its shared memory
    if (split > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    float zt = 0.f;  // the target's logit, on its way while the row is read
    if (rank == 0 && tid == 0 && logp) {
        int tgt = targets[row];
        if (tgt < 0 || tgt >= V) {
            set_status(status, GPT2_FLAG_TARGET_RANGE);
            tgt = 0;
        }
        zt = to_float(z[tgt]);
    }

    Stats x = {-INFINITY, 0.f, 0.f};
    int i = v0 + tid;
    for (const int whole = min(v1, V / VEC<T>); i + (BATCH - 1) * NT < whole; i += BATCH * NT) {
        uint4 u[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; b++) u[b] = __ldg(zv + i + b * NT);
        add_batch<T>(u, x);
    }
    {  // the rest, BATCH vectors at most, with the one that V cuts
        uint4 u[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; b++)
            if (i + b * NT < v1) u[b] = __ldg(zv + i + b * NT);
#pragma unroll
        for (int b = 0; b < BATCH; b++)
            if (i + b * NT < v1) add_vector<T>(u[b], i + b * NT, V, x);
    }
    const float mine = x.m;  // this thread's largest logit
    x = join<32>(x);
    if (lane == 0) ws[tid >> 5] = x;
    if (split > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    static_assert(NT / 32 <= 8 && MAX_SPLIT == 8, "eight lanes join the warps, and the blocks");
    const Stats empty = {-INFINITY, 0.f, 0.f};
    auto finish = [&](const Stats& r) {  // by the first warp
        if (lane) return;
        const Row w(r);
        lse[row] = w.lse();
        if (entropy) entropy[row] = w.entropy(r);
        if (logp) logp[row] = w.logp(zt);
        whole[0] = w.m, whole[1] = w.ln_s;
    };
    auto meet = [&] {  // the warps' sums, by the first warp
        if (tid >= 32) return;
        x = join<8>(lane < NT / 32 ? ws[lane] : empty);
        if (split == 1) finish(x);
        else if (lane == 0) *cg::this_cluster().map_shared_rank(&cs[rank], 0) = x;
    };
    if constexpr (!TOP) {
        __syncthreads();
        meet();
    }

    if constexpr (TOP) {
        static_assert(NT >= 4 * MAX_K && CAND == 2 * NT, "the sizes below");
        // The k-th largest of the maxima of 64 groups of four threads (of the threads, where fewer than 2 k groups have
        // data) bounds the k-th largest logit from below. -inf and no data come out as the lowest.
        const bool any = v0 + tid < v1;
        const uint32_t key = any ? (uint32_t)(order_key(mine, 0) >> 32) : 0;
        const bool fours = min(NT, v1 - v0) >= 8 * k;
        const int groups = fours ? NT / 4 : NT;
        uint32_t most = key;
        if (fours) {
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        }
        if (!fours) maxima[tid] = most;
        else if (lane % 4 == 0) maxima[tid / 4] = most;
        if (tid == 0) bound = ~0u, count = 0;
        __syncthreads();
        meet();
        if (NT - 1 - tid < groups) {  // (the last warps: the first is busy)
            const uint32_t own = maxima[NT - 1 - tid];
            int above = 0;
            for (int j = 0; j < groups; j += 4) {
                const uint4 o = *reinterpret_cast<const uint4*>(maxima + j);
                above += (o.x > own) + (o.y > own) + (o.z > own) + (o.w > own);
            }
            if (above < k) atomicMin(&bound, own);
        }
        __syncthreads();
        const uint32_t least = bound;
        auto each = [&](auto&& f) {  // this thread's logits as keys
            for (int v = v0 + tid; v < v1; v += NT) {
                float g[VEC<T>];
                unpack(__ldg(zv + v), g);
#pragma unroll
                for (int j = 0; j < VEC<T>; j++)
                    if (v * VEC<T> + j < V) f(order_key(g[j], v * VEC<T> + j));
            }
        };
        // The logits that reach the bound: the vectors of each thread whose maximum does, by its whole warp, one to a
        // lane, four threads' at a time. Where many are at the bound (more than CAND, or half a warp's threads), those
        // above it, and the first columns at it after them.
        constexpr int HOT = 4;
        bool equal = false;
        for (uint32_t from = least;; from++) {
            uint32_t hot = __ballot_sync(0xffffffffu, any && key >= from);
            if (!equal && __popc(hot) > 16) {
                hot = 0;
                if (lane == 0) atomicAdd(&count, CAND + 1);
            }
            while (hot) {
                int v[HOT];
#pragma unroll
                for (int h = 0; h < HOT; h++) {
                    v[h] = hot ? v0 + (tid & ~31) + __ffs(hot) - 1 + lane * NT : v1;
                    hot &= hot - 1;
                }
                while (__any_sync(0xffffffffu, min(min(v[0], v[1]), min(v[2], v[3])) < v1)) {
                    uint4 u[HOT];
#pragma unroll
                    for (int h = 0; h < HOT; h++)
                        if (v[h] < v1) u[h] = __ldg(zv + v[h]);
#pragma unroll
                    for (int h = 0; h < HOT; h++) {
                        if (v[h] >= v1) continue;
                        float g[VEC<T>];
                        unpack(u[h], g);
#pragma unroll
                        for (int j = 0; j < VEC<T>; j++) {
                            const uint64_t q = order_key(g[j], v[h] * VEC<T> + j);
                            if ((uint32_t)(q >> 32) >= from && v[h] * VEC<T> + j < V) {
                                const int at = atomicAdd(&count, 1);
                                if (at < CAND) keys[at] = q;
                            }
                        }
                        v[h] += 32 * NT;
                    }
                }
            }
            __syncthreads();
            if (equal || count <= CAND) break;
            equal = true;
            __syncthreads();
            if (tid == 0) count = 0;
            __syncthreads();
        }
        uint64_t* list = keys;
        if (split > 1) list = cg::this_cluster().map_shared_rank(lists, 0) + rank * MAX_K;
        const int n = count;
        if (n <= CAND) {
            uint64_t q[2];
            int r[2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int c = tid + h * NT;
                q[h] = c < n ? keys[c] : 0;
                r[h] = MAX_K;
                if (c < n) {
                    r[h] = 0;
                    for (int j = 0; j < n; j++) r[h] += keys[j] > q[h];
                }
            }
            __syncthreads();
#pragma unroll
            for (int h = 0; h < 2; h++)
                if (r[h] < k) list[r[h]] = q[h];
            if (tid < 32) {
                int have = min(n, k);
                if (equal) have = add_equal<T>(zv, v0, v1, V, least, have, k, list);
                for (int c = have + lane; c < k; c += 32) list[c] = 0;  // a part with fewer than k columns
            }
        } else {
            // one by one: the largest of the threads' largest, whose thread then looks for its next
            uint64_t best = 0;
            each([&](uint64_t q) { best = q > best ? q : best; });
            uint64_t found[(MAX_K + NT - 1) / NT] = {0};
            for (int r = 0; r < k; r++) {
                __syncthreads();
                keys[tid] = best;
                __syncthreads();
                uint64_t top = 0;
                for (int j = lane; j < NT; j += 32) top = keys[j] > top ? keys[j] : top;
#pragma unroll
                for (int o = 16; o > 0; o /= 2) {
                    const uint64_t y = __shfl_xor_sync(0xffffffffu, top, o);
                    top = y > top ? y : top;
                }
                if (tid == r) found[0] = top;
                if (best == top && top) {
                    best = 0;
                    each([&](uint64_t q) { best = q < top && q > best ? q : best; });
                }
            }
            __syncthreads();
            if (tid < MAX_K && (tid < k || split > 1)) list[tid] = tid < k ? found[0] : 0;
        }
    }
    if (split > 1) {
        cg::this_cluster().sync();
        if (rank) return;
        if (tid < 32) finish(join<8>(lane < split ? cs[lane] : empty));
    }
    if constexpr (TOP) {
        if (split > 1) {  // the k largest of the parts' lists
            for (int c = tid; c < split * MAX_K; c += NT) {
                const uint64_t q = lists[c];
                if (!q || (c % MAX_K) >= k) continue;
                int r = c % MAX_K;  // its own list is sorted
                for (int s = 0; s < split; s++)
                    if (s != c / MAX_K)
                        for (int j = 0; j < k && lists[s * MAX_K + j] > q; j++) r++;
                if (r < k) keys[r] = q;
            }
        }
        __syncthreads();
        if (tid < k) {
            const uint64_t q = keys[tid];
            top_ids[(int64_t)row * k + tid] = key_col(q);
            top_logp[(int64_t)row * k + tid] = Row(whole[0], whole[1]).logp(key_logit(q));
        }
    }
}

// Many rows with alternatives: the search for them is a few microseconds of
// waiting, so eight warps read row after row and two others search the rows
// before: they are handed each reading thread's largest logit and the warps'
// sums through shared memory. A block for a row that read and then searched
// took 59 us for 2043 rows of 50257 with 20 alternatives and 734 for 32768,
// this 51 and 686; three places for a thread's batches instead of two took 70
// (the search's own loads wait behind them).
constexpr int TNT = 256;   // threads that read
constexpr int TB = 4;      // vectors of its batch
constexpr int TOP_BLOCKS = 3;  // on an SM
constexpr int RING = 2;    // batches that a reading thread has in shared memory or on their way
constexpr int LOOK = 16;   // threads whose vectors the search has in shared memory at once, 32 of each
constexpr int LIST = 256;  // candidates that fit (all logits of a row with fewer than 32 vectors)
constexpr int MANY = 128;  // of the reading threads reach the bound: equal logits (k threads, or k groups of four, else)
struct Search {            // a searching warp's own
    uint4 part[LOOK][32];
    uint64_t keys[LIST], out[MAX_K];
    int hot[TNT], vectors[LIST], found, count;
};
struct TopShared {
    uint4 ring[RING][TB][TNT];
    Search search[2];
    Stats ws[2][TNT / 32];
    uint32_t maxima[2][TNT];  // a thread's largest logit (the lowest: -inf, or none)
};
// Hardware barriers of the reading threads and the search, a pair for each place: its row is read; its row is done with.
__device__ __forceinline__ void full_sync(int b) {
    if (b) asm volatile("bar.sync 2, %0;" ::"n"(TNT + 32) : "memory");
    else asm volatile("bar.sync 1, %0;" ::"n"(TNT + 32) : "memory");
}
__device__ __forceinline__ void full_arrive(int b) {
    if (b) asm volatile("bar.arrive 2, %0;" ::"n"(TNT + 32) : "memory");
    else asm volatile("bar.arrive 1, %0;" ::"n"(TNT + 32) : "memory");
}
__device__ __forceinline__ void empty_sync(int b) {
    if (b) asm volatile("bar.sync 4, %0;" ::"n"(TNT + 32) : "memory");
    else asm volatile("bar.sync 3, %0;" ::"n"(TNT + 32) : "memory");
}
__device__ __forceinline__ void empty_arrive(int b) {
    if (b) asm volatile("bar.arrive 4, %0;" ::"n"(TNT + 32) : "memory");
    else asm volatile("bar.arrive 3, %0;" ::"n"(TNT + 32) : "memory");
}

template <typename T>
__global__ void __launch_bounds__(TNT + 64, TOP_BLOCKS)
    logprobs_top_kernel(float* __restrict__ logp, float* __restrict__ lse, float* __restrict__ entropy,
                        float* __restrict__ top_logp, int32_t* __restrict__ top_ids, int k,
                        const T* __restrict__ logits, const int32_t* __restrict__ targets, int N, int V, int Vp,
                        int* status) {
    extern __shared__ __align__(16) uint8_t smem[];
    TopShared& sh = *reinterpret_cast<TopShared*>(smem);
    auto& maxima = sh.maxima;
    auto& ws = sh.ws;
    const int tid = threadIdx.x, lane = tid & 31, nv = (V + VEC<T> - 1) / VEC<T>;
    if (tid < TNT) {
        // a thread copies and reads its own vectors, across the ends of rows
        int64_t next = blockIdx.x;  // the row and the first vector of the batch to be asked for next
        int at = tid, slot = 0;
        auto ask = [&](int to) {
            if (next < N) {
                const uint4* zv = reinterpret_cast<const uint4*>(logits + next * Vp);
#pragma unroll
                for (int e = 0; e < TB; e++)
                    if (at + e * TNT < nv) cp_async16(&sh.ring[to][e][tid], zv + at + e * TNT);
                at += TB * TNT;
                if (at - tid >= nv) at = tid, next += gridDim.x;
            }
            cp_async_commit();
        };
#pragma unroll
        for (int r = 0; r < RING - 1; r++) ask(r);
        int it = 0;
        for (int64_t row = blockIdx.x; row < N; row += gridDim.x, it++) {
            const int b = it & 1;
            Stats x = {-INFINITY, 0.f, 0.f};
            for (int v = tid; v - tid < nv; v += TB * TNT) {
                ask(slot == 0 ? RING - 1 : slot - 1);
                cp_async_wait<RING - 1>();
                if (v + (TB - 1) * TNT < V / VEC<T>) {
                    uint4 u[TB];
#pragma unroll
                    for (int e = 0; e < TB; e++) u[e] = sh.ring[slot][e][tid];
                    add_batch<T>(u, x);
                } else {
#pragma unroll 1
                    for (int e = 0; e < TB; e++)
                        if (v + e * TNT < nv) add_vector<T>(sh.ring[slot][e][tid], v + e * TNT, V, x);
                }
                slot = slot == RING - 1 ? 0 : slot + 1;
            }
            const uint32_t key = tid < nv ? (uint32_t)(order_key(x.m, 0) >> 32) : 0;
            x = join<32>(x);
            if (it >= 2) empty_sync(b);
            maxima[b][tid] = key;
            if (lane == 0) ws[b][tid >> 5] = x;
            full_arrive(b);
        }
        cp_async_wait<0>();
        return;
    }
    const int b = (tid - TNT) / 32;  // two warps search, every other row
    Search& mine = sh.search[b];
    for (int64_t row = blockIdx.x + (int64_t)b * gridDim.x; row < N; row += 2 * gridDim.x) {
        const T* z = logits + row * Vp;
        const uint4* zv = reinterpret_cast<const uint4*>(z);
        float zt = 0.f;
        if (logp && lane == 0) {
            int tgt = targets[row];
            if (tgt < 0 || tgt >= V) {
                set_status(status, GPT2_FLAG_TARGET_RANGE);
                tgt = 0;
            }
            zt = to_float(z[tgt]);
        }
        full_sync(b);
        const Stats empty = {-INFINITY, 0.f, 0.f};
        const Stats x = join<8>(lane < TNT / 32 ? ws[b][lane] : empty);
        Row w(x);
        if (lane == 0) {
            lse[row] = w.lse();
            if (entropy) entropy[row] = w.entropy(x);
            if (logp) logp[row] = w.logp(zt);
        }
        w = Row(__shfl_sync(0xffffffffu, w.m, 0), __shfl_sync(0xffffffffu, w.ln_s, 0));
        // The bound as above.
        uint32_t least = ~0u;
        if (min(TNT, nv) >= 8 * k) {
            static_assert(TNT == 256, "two groups of four threads to a lane");
            uint32_t own[2];
            int above[2] = {0, 0};
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int g = lane + 32 * h;
                const uint4 o = *reinterpret_cast<const uint4*>(&maxima[b][4 * g]);
                own[h] = max(max(o.x, o.y), max(o.z, o.w));
            }
#pragma unroll
            for (int j = 0; j < 32; j++) {
                const uint32_t o0 = __shfl_sync(0xffffffffu, own[0], j), o1 = __shfl_sync(0xffffffffu, own[1], j);
                above[0] += (o0 > own[0]) + (o1 > own[0]);
                above[1] += (o0 > own[1]) + (o1 > own[1]);
            }
            if (above[0] < k) least = own[0];
            if (above[1] < k) least = min(least, own[1]);
        } else {
            uint32_t own[TNT / 32];
            int above[TNT / 32];
#pragma unroll
            for (int h = 0; h < TNT / 32; h++) own[h] = maxima[b][lane + 32 * h], above[h] = 0;
            for (int j = 0; j < TNT; j += 4) {
                const uint4 o = *reinterpret_cast<const uint4*>(&maxima[b][j]);
#pragma unroll
                for (int h = 0; h < TNT / 32; h++)
                    above[h] += (o.x > own[h]) + (o.y > own[h]) + (o.z > own[h]) + (o.w > own[h]);
            }
#pragma unroll
            for (int h = 0; h < TNT / 32; h++)
                if (above[h] < k) least = min(least, own[h]);
        }
        least = __reduce_min_sync(0xffffffffu, least);
        uint32_t most[TNT / 32];
#pragma unroll
        for (int h = 0; h < TNT / 32; h++) most[h] = lane + 32 * h < nv ? maxima[b][lane + 32 * h] : 0;
        __syncwarp();
        if (row + 2 * gridDim.x < N) empty_arrive(b);  // their sums and maxima are read
        // The reading threads whose maximum reaches a bound.
        auto threads = [&](uint32_t bound) {
            int n = 0;
            __syncwarp();
#pragma unroll
            for (int h = 0; h < TNT / 32; h++) {
                const uint32_t vote = __ballot_sync(0xffffffffu, most[h] >= bound && lane + 32 * h < nv);
                if (vote >> lane & 1) mine.hot[n + __popc(vote & ((1u << lane) - 1))] = lane + 32 * h;
                n += __popc(vote);
            }
            if (lane == 0) mine.found = mine.count = 0;
            __syncwarp();
            return n;
        };
        // The first nh threads' logits that reach it, in any order: their number, or more than LIST.
        auto collect = [&](int nh, uint32_t bound) {
            // their vectors, copied at once, then looked at: those whose largest reaches the bound
            for (int h0 = 0; h0 < nh; h0 += LOOK)
                for (int at = 0; at * TNT < nv; at += 32) {
                    const int hn = min(LOOK, nh - h0), v0 = (at + lane) * TNT;
                    for (int h = 0; h < hn; h++) {
                        const int v = v0 + mine.hot[h0 + h];
                        if (v < nv) cp_async16(&mine.part[h][lane], zv + v);
                    }
                    cp_async_commit();
                    cp_async_wait<0>();
                    for (int h = 0; h < hn; h++) {
                        const int v = v0 + mine.hot[h0 + h];
                        if (v >= nv) continue;
                        float g[VEC<T>], top = -INFINITY;
                        unpack(mine.part[h][lane], g);
                        if (v == nv - 1) {
#pragma unroll
                            for (int j = 0; j < VEC<T>; j++)
                                if (v * VEC<T> + j >= V) g[j] = -INFINITY;
                        }
#pragma unroll
                        for (int j = 0; j < VEC<T>; j += 2) top = max_nan(top, g[j], g[j + 1]);
                        if ((uint32_t)(order_key(top, 0) >> 32) >= bound) {
                            const int to = atomicAdd(&mine.found, 1);
                            if (to < LIST) mine.vectors[to] = v;
                        }
                    }
                }
            __syncwarp();
            // and of these the logits that reach it
            const int nf = mine.found;
            if (nf > LIST) return nf;
            for (int c = lane; c < nf; c += 32) {
                const int v = mine.vectors[c];
                float g[VEC<T>];
                unpack(__ldg(zv + v), g);
#pragma unroll
                for (int j = 0; j < VEC<T>; j++) {
                    const uint64_t q = order_key(g[j], v * VEC<T> + j);
                    if ((uint32_t)(q >> 32) >= bound && v * VEC<T> + j < V) {
                        const int to = atomicAdd(&mine.count, 1);
                        if (to < LIST) mine.keys[to] = q;
                    }
                }
            }
            __syncwarp();
            return mine.count;
        };
        int nh = threads(least), n = nh <= MANY ? collect(nh, least) : LIST + 1;
        const bool equal = n > LIST;  // many at the bound: those above it first, then the first columns at it
        if (equal) {
            nh = threads(least + 1);
            n = collect(nh, least + 1);
        }
        if (n <= LIST) {
            for (int c = lane; c < n; c += 32) {
                const uint64_t q = mine.keys[c];
                int r = 0;
                for (int j = 0; j < n; j++) r += mine.keys[j] > q;
                if (r < k) mine.out[r] = q;
            }
            if (equal) add_equal<T>(zv, 0, nv, V, least, n, k, mine.out);
        } else {
            // many in few threads: one by one, each the largest of the reading threads' largest, whose vectors are
            // then looked through for the next
            auto best_of = [&](int t, uint64_t below) {
                uint64_t best = 0;
                for (int v = t + lane * TNT; v < nv; v += 32 * TNT) {
                    float g[VEC<T>];
                    unpack(__ldg(zv + v), g);
#pragma unroll
                    for (int j = 0; j < VEC<T>; j++) {
                        const uint64_t q = order_key(g[j], v * VEC<T> + j);
                        if (v * VEC<T> + j < V && q < below && q > best) best = q;
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o /= 2) {
                    const uint64_t y = __shfl_xor_sync(0xffffffffu, best, o);
                    best = y > best ? y : best;
                }
                return best;
            };
            static_assert(LIST >= TNT, "the largest of each reading thread");
            __syncwarp();
            for (int t = 0; t < TNT; t++) {
                const uint64_t best = best_of(t, ~0ull);
                if (lane == 0) mine.keys[t] = best;
            }
            for (int r = 0; r < k; r++) {
                __syncwarp();
                uint64_t top = 0;
                for (int t = lane; t < TNT; t += 32) top = mine.keys[t] > top ? mine.keys[t] : top;
#pragma unroll
                for (int o = 16; o > 0; o /= 2) {
                    const uint64_t y = __shfl_xor_sync(0xffffffffu, top, o);
                    top = y > top ? y : top;
                }
                const int t = key_col(top) / VEC<T> % TNT;
                const uint64_t next = best_of(t, top);
                __syncwarp();
                if (lane == 0) mine.out[r] = top, mine.keys[t] = next;
            }
        }
        __syncwarp();
        for (int r = lane; r < k; r += 32) {
            const uint64_t q = mine.out[r];
            top_ids[row * k + r] = key_col(q);
            top_logp[row * k + r] = w.logp(key_logit(q));
        }
        __syncwarp();
    }
}

// Row blockIdx.x, vectors part blockIdx.y of gridDim.y.
constexpr int BNT = 256;
template <typename T>
__global__ void __launch_bounds__(BNT)
    logprobs_bwd_kernel(T* dlogits, const T* logits, const int32_t* __restrict__ targets,
                        const float* __restrict__ lse, const float* __restrict__ entropy,
                        const float* __restrict__ dlogp, const float* __restrict__ dlse,
                        const float* __restrict__ dentropy, int V, int Vp, int* status) {
    const int row = blockIdx.x;
    const uint4* zv = reinterpret_cast<const uint4*>(logits + (int64_t)row * Vp);
    uint4* dv = reinterpret_cast<uint4*>(dlogits + (int64_t)row * Vp);
    int v0, v1;
    part(Vp / VEC<T>, gridDim.y, blockIdx.y, v0, v1);
    const float L = lse[row], H = dentropy ? entropy[row] : 0.f;
    const float g = dlogp ? dlogp[row] : 0.f, b = dentropy ? dentropy[row] : 0.f;
    const float c = (dlse ? dlse[row] : 0.f) - g - b * H;  // dz = p (c - b log p) + g [target]
    int tgt = -1;
    if (dlogp) {
        tgt = targets[row];
        if (tgt < 0 || tgt >= V) {
            if (threadIdx.x == 0 && blockIdx.y == 0) set_status(status, GPT2_FLAG_TARGET_RANGE);
            tgt = 0;
        }
    }
    const bool none = L == -INFINITY;
    const int tvec = tgt < 0 ? -1 : tgt / VEC<T>;
    for (int i = v0 + (int)threadIdx.x; i < v1; i += BATCH * BNT) {
        uint4 u[BATCH];
#pragma unroll
        for (int e = 0; e < BATCH; e++)
            if (i + e * BNT < v1) u[e] = __ldcs(zv + i + e * BNT);
#pragma unroll
        for (int e = 0; e < BATCH; e++) {
            const int v = i + e * BNT;
            if (v >= v1) break;
            float f[VEC<T>];
            unpack(u[e], f);
#pragma unroll
            for (int j = 0; j < VEC<T>; j++) {
                const float lp = f[j] - L, p = ex2_approx(lp * LOG2E);
                f[j] = p * (c - b * fmaxf(lp, -1e4f));  // p is 0 long before the bound
            }
            if (v == tvec) {
#pragma unroll
                for (int j = 0; j < VEC<T>; j++)
                    if (v * VEC<T> + j == tgt) f[j] += g;
            }
            if (none || v * VEC<T> + VEC<T> > V) {
#pragma unroll
                for (int j = 0; j < VEC<T>; j++)
                    if (none || v * VEC<T> + j >= V) f[j] = 0.f;
            }
            uint4 w;
            pack(w, f);
            __stcs(dv + v, w);
        }
    }
}

template <typename T, int NT, bool TOP>
int forward(float* logp, float* lse, float* entropy, float* top_logp, int32_t* top_ids, int k, const T* logits,
            const int32_t* targets, int N, int V, int Vp, int* status, cudaStream_t s) {
    // as many blocks to a row as leave each SM one, and each thread a vector (8 rows of 50257 in fp32: 6.2 us with
    // eight, 8.3 with one; with 5 alternatives 8.5 with four, 11.3 with eight, with 40 16.5 and 32)
    int split = 1;
    while (split < (TOP ? TOP_SPLIT : MAX_SPLIT) && (int64_t)N * split * 2 <= gpt2_num_sms() && V / VEC<T> >= split * 2 * 256) split *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(N * split));
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = split;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = split > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, logprobs_kernel<T, NT, TOP>, logp, lse, entropy, top_logp, top_ids, k, logits, targets,
                           V, Vp, split, status) != cudaSuccess)
        return GPT2_ERR_CUDA;
    return 1;
}
template <typename T>
int forward_top(float* logp, float* lse, float* entropy, float* top_logp, int32_t* top_ids, int k, const T* logits,
                const int32_t* targets, int N, int V, int Vp, int* status, cudaStream_t s) {
    const void* kernel = (const void*)logprobs_top_kernel<T>;
    if (smem_attr(kernel, sizeof(TopShared)) != cudaSuccess) return GPT2_ERR_CUDA;
    logprobs_top_kernel<T><<<min(N, TOP_BLOCKS * gpt2_num_sms()), TNT + 64, sizeof(TopShared), s>>>(
        logp, lse, entropy, top_logp, top_ids, k, logits, targets, N, V, Vp, status);
    return 1;
}
// Threads of a block: twice as many rows on their way in blocks of 128 read
// 32768 rows of 50257 at the speed of a copy (498 us; about 8% more with 256), but few
// rows want the wider block. With alternatives, rows are handed to searching
// warps where a block for each (four to an SM) would come in more than one
// round, and for k up to 32 (rows of 50257 with 20: 600 take 25 us handed over
// and 18 a block each, 1000 31 either way, 2043 51 and 59; 8192 rows of 32768
// with 20 142 and 158, with 64 331 and 264).
template <typename T, typename... A>
int forward_of(int k, int N, A... args) {
    const int sms = gpt2_num_sms();
    if (k) return k <= 32 && N > 4 * sms ? forward_top<T>(args...) : forward<T, 256, true>(args...);
    return N > sms ? forward<T, 128, false>(args...) : forward<T, 256, false>(args...);
}

template <typename T>
int backward(T* dlogits, const T* logits, const int32_t* targets, const float* lse, const float* entropy,
             const float* dlogp, const float* dlse, const float* dentropy, int N, int V, int Vp, int* status,
             cudaStream_t s) {
    int split = 1;
    while ((int64_t)N * split < 4 * gpt2_num_sms() && Vp / VEC<T> > split * BATCH * BNT) split *= 2;
    logprobs_bwd_kernel<T><<<dim3(N, split), BNT, 0, s>>>(dlogits, logits, targets, lse, entropy, dlogp, dlse, dentropy,
                                                         V, Vp, status);
    return 1;
}

}  // namespace

int launch_token_logprobs(int dtype, float* logp, float* lse, float* entropy, float* top_logp, int32_t* top_ids,
                          int k, const void* logits, const int32_t* targets, int N, int V, int Vp, int* status,
                          cudaStream_t s) {
    if (dtype == GPT2_MODE_BF16)
        return forward_of<bf16>(k, N, logp, lse, entropy, top_logp, top_ids, k, (const bf16*)logits, targets, N, V, Vp,
                                status, s);
    return forward_of<float>(k, N, logp, lse, entropy, top_logp, top_ids, k, (const float*)logits, targets, N, V, Vp,
                             status, s);
}

int launch_token_logprobs_backward(int dtype, void* dlogits, const void* logits, const int32_t* targets,
                                   const float* lse, const float* entropy, const float* dlogp, const float* dlse,
                                   const float* dentropy, int N, int V, int Vp, int* status, cudaStream_t s) {
    if (dtype == GPT2_MODE_BF16)
        return backward((bf16*)dlogits, (const bf16*)logits, targets, lse, entropy, dlogp, dlse, dentropy, N, V, Vp,
                        status, s);
    return backward((float*)dlogits, (const float*)logits, targets, lse, entropy, dlogp, dlse, dentropy, N, V, Vp,
                    status, s);
}
