// Packed causal attention with grouped heads in fp32 (the exact-parity mode):
// fp32 FMA throughout, bound by it.
//
// Rows are a key head's queries x the heads of its group, in this order, so
// shared heads share the K and V blocks (and their sums dK, dV lie inside the
// products). A block of 256 threads takes 64 rows (forward, dQ) or 64 keys
// (dK, dV) against blocks of 64 of the others, all in shared memory; thread
// (ty, tx) of 16 x 16 holds rows ty + 16 r and columns tx + 16 c of the 64 x 64
// scores. Scores are dot products over 16-byte pieces of both rows, products
// with P or dS walk 16-byte pieces of a P row: either way 8 shared 16-byte
// loads feed 64 FMA a thread, and the row padding of four floats spreads the
// rows that a warp reads at once over the banks. (128 threads with twice the
// columns load a quarter less and took as long.) The forward's tiles are sorted,
// the longest first, where they come in several rounds: 16 documents of 3582
// tokens and 12 heads take 78 us (unsorted 91), of which the FMA of the tiles,
// the masked halves of the diagonal ones included, are 33 and all instructions
// 51. Gradients have one writer each: deterministic.
#include "attention_packed.cuh"

namespace {

constexpr int TL = 64, NT = 256;
constexpr int TX = 16, NC = TL / TX, NR = 4;  // threads of a row, their columns; rows of a thread
constexpr int LP = TL + 4;  // floats of a P row
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct Args {
    PackedAttn a;
    PackedAttnGrad g;
    int group;
    const PackedPlan* plan;  // forward: its tiles, or null
    int key_blocks;  // backward: the blocks of dK, dV, before those of dQ
    float scale, scale_log2;
};

template <int HD> struct Shape {
    static constexpr int LD = HD + 4;  // floats of an operand's row
    static constexpr int DV = HD / TX > 1 ? HD / TX : 1;  // output columns of a thread
    static constexpr int T = TL * LD;  // floats of a tile
    // output column of element e (HD 8: the upper half of the threads doubles the lower)
    static __device__ __forceinline__ int col(int tx, int e) { return HD < TX ? tx % HD : tx * DV + e; }
    static __device__ __forceinline__ bool writes(int tx) { return HD >= TX || tx < HD; }
};

// Rows [0, n) of a tile from src(row), the rest zero.
template <int HD, typename F> __device__ __forceinline__ void load_tile(float* dst, int n, F src) {
    constexpr int C = HD / 4;
    for (int i = threadIdx.x; i < TL * C; i += NT) {
        const int r = i / C, c = i % C;
        const float* p = src(r < n ? r : 0) + c * 4;
        const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst + r * Shape<HD>::LD + c * 4);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(p), "r"(r < n ? 16 : 0) : "memory");
    }
    cp_async_commit();
}

// s[r][c] = A row (ty + 16 r) . B row (tx + 16 c)
template <int HD> __device__ __forceinline__ void dots(float (&s)[NR][NC], const float* A, const float* B, int ty, int tx) {
    constexpr int LD = Shape<HD>::LD;
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
        for (int c = 0; c < NC; c++) s[r][c] = 0.f;
#pragma unroll 4
    for (int d = 0; d < HD; d += 4) {
        float4 x[NR], y[NC];
#pragma unroll
        for (int r = 0; r < 4; r++) x[r] = *reinterpret_cast<const float4*>(A + (ty + 16 * r) * LD + d);
#pragma unroll
        for (int c = 0; c < NC; c++) y[c] = *reinterpret_cast<const float4*>(B + (tx + TX * c) * LD + d);
#pragma unroll
        for (int r = 0; r < 4; r++)
#pragma unroll
            for (int c = 0; c < NC; c++)
                s[r][c] = fmaf(x[r].w, y[c].w, fmaf(x[r].z, y[c].z, fmaf(x[r].y, y[c].y, fmaf(x[r].x, y[c].x, s[r][c]))));
    }
}

// o[r][e] += P row (ty + 16 r) . column col(e) of B
template <int HD>
__device__ __forceinline__ void products(float (&o)[4][Shape<HD>::DV], const float* P, const float* B, int ty, int tx) {
    constexpr int LD = Shape<HD>::LD, DV = Shape<HD>::DV;
#pragma unroll 4
    for (int j = 0; j < TL; j += 4) {
        float p[4][4];
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const float4 v = *reinterpret_cast<const float4*>(P + (ty + 16 * r) * LP + j);
            p[r][0] = v.x, p[r][1] = v.y, p[r][2] = v.z, p[r][3] = v.w;
        }
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const float* b = B + (j + k) * LD;
            float v[DV];
            if constexpr (DV == 4) {
                *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(b + Shape<HD>::col(tx, 0));
            } else if constexpr (DV == 2) {
                *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(b + Shape<HD>::col(tx, 0));
            } else {
#pragma unroll
                for (int e = 0; e < DV; e++) v[e] = b[Shape<HD>::col(tx, e)];
            }
#pragma unroll
            for (int r = 0; r < 4; r++)
#pragma unroll
                for (int e = 0; e < DV; e++) o[r][e] = fmaf(p[r][k], v[e], o[r][e]);
        }
    }
}
__device__ __forceinline__ void put(float* P, const float (&s)[NR][NC], int ty, int tx) {
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
        for (int c = 0; c < NC; c++) P[(ty + 16 * r) * LP + tx + TX * c] = s[r][c];
}
// Over the threads of a row.
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = TX / 2; o > 0; o /= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = TX / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Row i of a sequence and key head: query i / group, head i % group.
struct Rows {
    int q0, group, head0;
    __device__ __forceinline__ const float* at(const void* base, int64_t stride, int hd, int i) const {
        const int q = i / group;
        return (const float*)base + (int64_t)(q0 + q) * stride + (head0 + i - q * group) * hd;
    }
    __device__ __forceinline__ int64_t stat(int total_q, int i) const {  // index of lse, D
        const int q = i / group;
        return (int64_t)(head0 + i - q * group) * total_q + q0 + q;
    }
};

// Up to TL rows of a key head: rows at .. at + n - 1 from query q0 on, the keys of their sequence, and how many of
// those query q0 sees.
struct RowTile {
    int kh, q0, at, n, k0, lk, sees;
    __device__ __forceinline__ int keys(int i, int group) const { return max(0, min(lk, (at + i) / group + sees)); }
};
// The tile of a block of `blocks`; false for none.
__device__ __forceinline__ bool row_tile(const Args& A, int block, int blocks, RowTile& t) {
    const PackedAttn& a = A.a;
    const int slots = blocks / a.Hkv, i = block / a.Hkv;
    t.kh = block - i * a.Hkv;
    if (A.plan) {  // the longest tiles first
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (i >= A.plan->count) return false;
        const PackedTile p = A.plan->tile[i];
        t.q0 = p.r0, t.at = 0, t.n = p.n * A.group, t.k0 = p.s0, t.lk = p.len, t.sees = p.shift;
        return true;
    }
    const int slot = slots - 1 - i;  // the later rows of a sequence, which see more keys, first
    int first;
    const int s = find_slot(a.cu_q, a.n_seq, a.total_q, TL, slot, first, A.group);
    if (s < 0) return false;
    const PackedSeq p = packed_seq(a, s);
    t.q0 = p.q0, t.at = (slot - first) * TL, t.n = min(TL, p.lq * A.group - t.at);
    t.k0 = p.k0, t.lk = p.lk, t.sees = 1 + p.lk - p.lq;
    return t.at >= 0 && t.n > 0;  // (before 0: offsets that descend)
}

__global__ void __launch_bounds__(1024) packed_plan_f32_kernel(PackedAttn a, PackedCut cut, PackedPlan* plan) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    packed_plan_block(a, cut, plan, true);
}

template <int HD> __global__ void __launch_bounds__(NT) packed_fwd_f32_kernel(const __grid_constant__ Args A) {
    using S = Shape<HD>;
    const PackedAttn& a = A.a;
    extern __shared__ __align__(16) float sm[];
    float *sq = sm, *sk = sm + S::T, *sv = sk + S::T, *sp = sv + S::T;
    const int tid = threadIdx.x, tx = tid % TX, ty = tid / TX;
    if (blockIdx.x == 0 && !A.plan) packed_check(a, tid, NT);
    RowTile p;
    if (!row_tile(A, blockIdx.x, gridDim.x, p)) return;
    const int kh = p.kh, at = p.at, n = p.n;
    const Rows rows = {p.q0, A.group, kh * A.group};
    load_tile<HD>(sq, n, [&](int r) { return rows.at(a.q, a.q_stride, HD, at + r); });
    int vis[4];  // keys that the row sees
#pragma unroll
    for (int r = 0; r < 4; r++) {
        const int i = ty + 16 * r;
        vis[r] = i < n ? p.keys(i, A.group) : 0;
    }
    const int keys = p.keys(n - 1, A.group);  // that any row sees
    float m[4], l[4], o[4][S::DV];
#pragma unroll
    for (int r = 0; r < 4; r++) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int e = 0; e < S::DV; e++) o[r][e] = 0.f;
    }
    auto load_k = [&](int j) {
        load_tile<HD>(sk, min(TL, keys - j), [&](int r) {
            return (const float*)a.k + (int64_t)(p.k0 + j + r) * a.k_stride + kh * HD;
        });
    };
    auto load_v = [&](int j) {
        load_tile<HD>(sv, min(TL, keys - j), [&](int r) {
            return (const float*)a.v + (int64_t)(p.k0 + j + r) * a.v_stride + kh * HD;
        });
    };
    if (keys > 0) load_k(0);
    for (int j = 0; j < keys; j += TL) {
        load_v(j);
        cp_async_wait<1>();  // K (and Q)
        __syncthreads();
        float s[NR][NC];
        dots<HD>(s, sq, sk, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; r++) {
            float mx = m[r];
#pragma unroll
            for (int c = 0; c < NC; c++) {
                s[r][c] = j + tx + TX * c < vis[r] ? s[r][c] * A.scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[r][c]);
            }
            mx = row_max(mx);
            const float f = m[r] == mx ? 1.f : ex2_approx(m[r] - mx), ref = mx == -INFINITY ? 0.f : mx;
            m[r] = mx;
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < NC; c++) {
                s[r][c] = ex2_approx(s[r][c] - ref);
                sum += s[r][c];
            }
            l[r] = l[r] * f + sum;
#pragma unroll
            for (int e = 0; e < S::DV; e++) o[r][e] *= f;
        }
        put(sp, s, ty, tx);
        cp_async_wait<0>();  // V
        __syncthreads();     // and every thread is done with K
        if (j + TL < keys) load_k(j + TL);
        products<HD>(o, sp, sv, ty, tx);
        __syncthreads();  // done with V and P
    }
    if (keys == 0) cp_async_wait<0>();  // Q, which nobody waited for
#pragma unroll
    for (int r = 0; r < 4; r++) {
        const int i = ty + 16 * r;
        const float sum = row_sum(l[r]), inv = vis[r] > 0 ? 1.f / sum : 0.f;
        if (i < n) {
            float* out = const_cast<float*>(rows.at(a.o, a.o_stride, HD, at + i));
#pragma unroll
            for (int e = 0; e < S::DV; e++)
                if (S::writes(tx)) out[S::col(tx, e)] = vis[r] > 0 ? o[r][e] * inv : 0.f;
            if (tx == 0) a.lse[rows.stat(a.total_q, at + i)] = vis[r] > 0 ? (m[r] + log2f(sum)) * LN2 : -INFINITY;
        }
    }
}

// dQ of 64 rows.
template <int HD> __device__ __forceinline__ void dq_rows(const Args& A, float* sm, int block, int blocks) {
    using S = Shape<HD>;
    const PackedAttn& a = A.a;
    float *sq = sm, *sy = sm + S::T, *sk = sy + S::T, *sv = sk + S::T, *sp = sv + S::T;
    const int tid = threadIdx.x, tx = tid % TX, ty = tid / TX;
    RowTile p;
    if (!row_tile(A, block, blocks, p)) return;
    const int kh = p.kh, at = p.at, n = p.n;
    const Rows rows = {p.q0, A.group, kh * A.group};
    load_tile<HD>(sq, n, [&](int r) { return rows.at(a.q, a.q_stride, HD, at + r); });
    load_tile<HD>(sy, n, [&](int r) { return rows.at(A.g.dout, A.g.dout_stride, HD, at + r); });
    int vis[4];
    float lse2[4], D[4], dq[4][S::DV];
    cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; r++) {
        const int i = ty + 16 * r;
        vis[r] = i < n ? p.keys(i, A.group) : 0;
        float d = 0.f;
        lse2[r] = 0.f;
        if (i < n) {
            const float* o = rows.at(a.o, a.o_stride, HD, at + i);
#pragma unroll
            for (int e = 0; e < S::DV; e++)
                if (S::writes(tx)) d += o[S::col(tx, e)] * sy[i * S::LD + S::col(tx, e)];
            if (vis[r] > 0) lse2[r] = a.lse[rows.stat(a.total_q, at + i)] * LOG2E;
        }
        D[r] = row_sum(d);
#pragma unroll
        for (int e = 0; e < S::DV; e++) dq[r][e] = 0.f;
    }
    const int keys = p.keys(n - 1, A.group);
    for (int j = 0; j < keys; j += TL) {
        const int nk = min(TL, keys - j);
        load_tile<HD>(sk, nk, [&](int r) { return (const float*)a.k + (int64_t)(p.k0 + j + r) * a.k_stride + kh * HD; });
        load_tile<HD>(sv, nk, [&](int r) { return (const float*)a.v + (int64_t)(p.k0 + j + r) * a.v_stride + kh * HD; });
        cp_async_wait<1>();
        __syncthreads();
        float s[NR][NC], dp[NR][NC];
        dots<HD>(s, sq, sk, ty, tx);
        cp_async_wait<0>();
        __syncthreads();
        dots<HD>(dp, sy, sv, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; r++)
#pragma unroll
            for (int c = 0; c < NC; c++)
                s[r][c] = j + tx + TX * c < vis[r] ? ex2_approx(fmaf(s[r][c], A.scale_log2, -lse2[r])) * (dp[r][c] - D[r])
                                                  : 0.f;
        put(sp, s, ty, tx);
        __syncthreads();
        products<HD>(dq, sp, sk, ty, tx);
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < 4; r++) {
        const int i = ty + 16 * r;
        if (i >= n) continue;
        float* out = const_cast<float*>(rows.at(A.g.dq, A.g.dq_stride, HD, at + i));
#pragma unroll
        for (int e = 0; e < S::DV; e++)
            if (S::writes(tx)) out[S::col(tx, e)] = dq[r][e] * A.scale;
    }
}

// dK, dV of 64 keys of one key head; D = rowsum(dO * O) of each block of rows
// on the way, so that nothing waits for dQ.
template <int HD> __device__ __forceinline__ void dkdv_keys(const Args& A, float* sm, int block) {
    using S = Shape<HD>;
    const PackedAttn& a = A.a;
    float *sk = sm, *sv = sm + S::T, *sq = sv + S::T, *sy = sq + S::T, *sp = sy + S::T, *sd = sp + TL * LP;
    float* stat = sd + TL * LP;  // lse log2(e), D of the block's rows
    const int tid = threadIdx.x, tx = tid % TX, ty = tid / TX;
    const int slot = block / a.Hkv, kh = block - slot * a.Hkv;
    int first;
    const int s0 = find_slot(a.cu_k, a.n_seq, a.total_k, TL, slot, first);
    if (s0 < 0) return;
    const PackedSeq p = packed_seq(a, s0);
    const int at = (slot - first) * TL;
    if (at < 0 || at >= p.lk) return;
    const Rows rows = {p.q0, A.group, kh * A.group};
    const int nk = min(TL, p.lk - at), off = p.lk - p.lq, all = p.lq * A.group;
    load_tile<HD>(sk, nk, [&](int r) { return (const float*)a.k + (int64_t)(p.k0 + at + r) * a.k_stride + kh * HD; });
    load_tile<HD>(sv, nk, [&](int r) { return (const float*)a.v + (int64_t)(p.k0 + at + r) * a.v_stride + kh * HD; });
    float dk[4][S::DV], dv[4][S::DV];
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
        for (int e = 0; e < S::DV; e++) dk[r][e] = dv[r][e] = 0.f;
    // the first row that sees the tile's first key
    for (int i = max(0, at - off) * A.group / TL * TL; i < all; i += TL) {
        const int n = min(TL, all - i);
        load_tile<HD>(sq, n, [&](int r) { return rows.at(a.q, a.q_stride, HD, i + r); });
        load_tile<HD>(sy, n, [&](int r) { return rows.at(A.g.dout, A.g.dout_stride, HD, i + r); });
        if (tid < TL) {
            const float v = tid < n ? a.lse[rows.stat(a.total_q, i + tid)] : 0.f;
            stat[tid] = v == -INFINITY ? 0.f : v * LOG2E;
        }
        constexpr int Q = HD / 4;  // four threads to a row of O
        const int drow = tid / 4, dcol = tid % 4 * Q;
        float o[Q];
#pragma unroll
        for (int e = 0; e < Q; e++) o[e] = 0.f;
        if (drow < n) {
            const float* x = rows.at(a.o, a.o_stride, HD, i + drow) + dcol;
#pragma unroll
            for (int e = 0; e < Q; e += 2) *reinterpret_cast<float2*>(o + e) = *reinterpret_cast<const float2*>(x + e);
        }
        cp_async_wait<0>();
        __syncthreads();
        float d = 0.f;
#pragma unroll
        for (int e = 0; e < Q; e++) d += o[e] * sy[drow * S::LD + dcol + e];
        d += __shfl_xor_sync(0xffffffffu, d, 1);
        d += __shfl_xor_sync(0xffffffffu, d, 2);
        if (tid % 4 == 0) stat[TL + drow] = d;
        float s[NR][NC], dp[NR][NC];
        dots<HD>(s, sk, sq, ty, tx);
        dots<HD>(dp, sv, sy, ty, tx);
        __syncthreads();  // D
#pragma unroll
        for (int c = 0; c < NC; c++) {
            const int row = tx + TX * c;
            // keys below this are seen
            const int seen = row < n ? (i + row) / A.group + 1 + off - at : 0;
            const float L = stat[row], D = stat[TL + row];
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const bool in = ty + 16 * r < seen;
                s[r][c] = in ? ex2_approx(fmaf(s[r][c], A.scale_log2, -L)) : 0.f;
                dp[r][c] = in ? s[r][c] * (dp[r][c] - D) : 0.f;
            }
        }
        put(sp, s, ty, tx);
        put(sd, dp, ty, tx);
        __syncthreads();
        products<HD>(dv, sp, sy, ty, tx);
        products<HD>(dk, sd, sq, ty, tx);
        __syncthreads();
    }
    cp_async_wait<0>();
#pragma unroll
    for (int r = 0; r < 4; r++) {
        const int j = ty + 16 * r;
        if (j >= nk) continue;
        const int64_t row = p.k0 + at + j;
        float* ok = (float*)A.g.dk + row * A.g.dk_stride + kh * HD;
        float* ov = (float*)A.g.dv + row * A.g.dv_stride + kh * HD;
#pragma unroll
        for (int e = 0; e < S::DV; e++) {
            if (!S::writes(tx)) continue;
            ok[S::col(tx, e)] = dk[r][e] * A.scale;
            ov[S::col(tx, e)] = dv[r][e];
        }
    }
}

// Both gradients in one launch, dQ beside dK and dV: 9 chunks of up to 400
// tokens (6 heads of 32 on 2), bound by the longest sequence's chain of tiles,
// take 29 us, one after the other 47.
template <int HD> __global__ void __launch_bounds__(NT) packed_bwd_f32_kernel(const __grid_constant__ Args A) {
    extern __shared__ __align__(16) float sm[];
    if (blockIdx.x == 0) packed_check(A.a, threadIdx.x, NT);
    if ((int)blockIdx.x < A.key_blocks) dkdv_keys<HD>(A, sm, blockIdx.x);
    else dq_rows<HD>(A, sm, blockIdx.x - A.key_blocks, gridDim.x - A.key_blocks);
}

Args args_of(const PackedAttn& a) {
    Args A = {};
    A.a = a;
    A.group = a.Hq / a.Hkv;
    A.scale = 1.f / sqrtf((float)a.hd);
    A.scale_log2 = LOG2E * A.scale;
    return A;
}
int row_blocks(const PackedAttn& a) {  // slots of the rows, times the key heads
    return (int)((int64_t)a.total_q * (a.Hq / a.Hkv) / TL + a.n_seq) * a.Hkv;
}

// The forward's sorted tiles of whole queries; with fewer blocks than are at work
// at once the sort would only be a launch more.
constexpr int SORT_BLOCKS = 2 * PACKED_SMS;
PackedCut row_cut(int Hq, int Hkv) { return PackedCut{false, max(1, TL / (Hq / Hkv)), TL}; }
size_t plan_bytes(int n_seq, int total_q, int Hq, int Hkv) {
    const int slots = packed_slots(total_q, n_seq, row_cut(Hq, Hkv).per);
    return Hq / Hkv <= TL && slots <= PACKED_PLAN_MAX && (int64_t)slots * Hkv > SORT_BLOCKS ? packed_plan_bytes(slots) : 0;
}

template <int HD> int forward(const PackedAttn& a, PackedPlan* plan, cudaStream_t s) {
    constexpr int SMEM = (3 * Shape<HD>::T + TL * LP) * 4;
    const auto kernel = packed_fwd_f32_kernel<HD>;
    if (smem_attr((const void*)kernel, SMEM) != cudaSuccess) return GPT2_ERR_CUDA;
    Args A = args_of(a);
    if (!plan_bytes(a.n_seq, a.total_q, a.Hq, a.Hkv)) {
        kernel<<<row_blocks(a), NT, SMEM, s>>>(A);
        return 1;
    }
    const PackedCut cut = row_cut(a.Hq, a.Hkv);
    A.plan = plan;
    packed_plan_f32_kernel<<<1, 1024, 0, s>>>(a, cut, plan);
    return launch_dependent(kernel, cut.slots(a) * a.Hkv, NT, SMEM, s, A) == cudaSuccess ? 2 : GPT2_ERR_CUDA;
}
template <int HD> int backward(const PackedAttn& a, const PackedAttnGrad& g, cudaStream_t s) {
    constexpr int SMEM = (4 * Shape<HD>::T + 2 * TL * LP + 2 * TL) * 4;  // (dQ uses less)
    const auto kernel = packed_bwd_f32_kernel<HD>;
    if (smem_attr((const void*)kernel, SMEM) != cudaSuccess) return GPT2_ERR_CUDA;
    Args A = args_of(a);
    A.g = g;
    A.key_blocks = a.total_k ? packed_slots(a.total_k, a.n_seq, TL) * a.Hkv : 0;
    kernel<<<A.key_blocks + (a.total_q ? row_blocks(a) : 0), NT, SMEM, s>>>(A);
    return 1;
}

}  // namespace

size_t attention_packed_forward_f32_scratch(int n_seq, int total_q, int Hq, int Hkv) {
    return plan_bytes(n_seq, total_q, Hq, Hkv);
}

int launch_attention_packed_forward_f32(const PackedAttn& a, PackedPlan* plan, cudaStream_t s) {
    switch (a.hd) {
        case 8: return forward<8>(a, plan, s);
        case 16: return forward<16>(a, plan, s);
        case 32: return forward<32>(a, plan, s);
        default: return forward<64>(a, plan, s);
    }
}

int launch_attention_packed_backward_f32(const PackedAttn& a, const PackedAttnGrad& g, cudaStream_t s) {
    switch (a.hd) {
        case 8: return backward<8>(a, g, s);
        case 16: return backward<16>(a, g, s);
        case 32: return backward<32>(a, g, s);
        default: return backward<64>(a, g, s);
    }
}
