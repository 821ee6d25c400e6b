// Packed attention forward for few queries (bf16, head size 64): at most 16
// rows (queries x heads of a group) per sequence and key head, one new token
// each above all. Bound by reading the keys and values once from HBM, so the
// products need only keep up: mma.sync on 16 rows, straight from registers.
//
// A block takes a part of one sequence's keys for one key head; its four warps
// take tiles of 32 keys in turn, each with its own running maximum, sum and
// output, and join at the end. Parts are of equal length whatever the
// sequence's, so ragged batches spread evenly; parts of one sequence are
// joined by a second kernel from scratch.
//
// A thread copies what it will use itself, 16 bytes at a time, into its own
// places in shared memory two tiles ahead (cp.async), so nothing is shared and
// nothing waits for other threads; loads into registers kept 34 KB in flight on
// an SM and 65% of the memory busy. The contraction's order is free as long as
// both sides agree, so a thread's 16 bytes are used as they come. Q K^T: thread (n = lane / 4, t = lane % 4) holds dims 8t .. 8t+7
// and 32+8t .. of key n, its 32-bit words being the fragments' (k, k+1) pairs,
// and of rows n, n + 8 of Q alike. P V: it holds dims 8n .. 8n+7 of keys 2t,
// 2t+1, 2t+8, 2t+9; byte permutes pair the keys, column n of the j-th product
// being dim 8n + j. So a warp reads whole 128-byte rows and a thread ends with
// 16 consecutive outputs of two rows.
#include "attention_packed.cuh"

namespace {

constexpr int HD = 64;
constexpr int WARPS = 4, TILE = 32;        // keys of a warp's tile
constexpr int STEP = WARPS * TILE;         // keys of a block's turn
constexpr int ROWS = 16;
constexpr int NST = 3;                     // tiles that a warp has in shared memory or on their way
constexpr int STAGE = 16 * 32 * 16;        // bytes of a tile: 16 pieces of 16 bytes for each lane
constexpr int SMEM = WARPS * NST * STAGE;
constexpr int PART = HD + 2;               // floats of a row's partial result: O, m, l
constexpr int FILL = 4 * 152;              // blocks that a call is cut into
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct Args {
    PackedAttn a;
    int group, keys;  // keys of a part
    int rows;         // rows of scratch per (part, key head)
    float scale_log2;
    float* scratch;   // [slot][key head][rows][PART]; a sequence's parts own the slots of its keys (find_slot)
};

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
// The factor from reference m to n >= m (0 from -inf; n = -inf only with m).
__device__ __forceinline__ float carry(float m, float n) { return m == n ? 1.f : ex2_approx(m - n); }

__global__ void __launch_bounds__(WARPS * 32) packed_few_kernel(const __grid_constant__ Args A) {
    const PackedAttn& a = A.a;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float sm[WARPS][ROWS], sl[WARPS][ROWS];
    float (*so)[ROWS][HD + 4] = reinterpret_cast<float (*)[ROWS][HD + 4]>(smem);  // once the tiles are done with
    static_assert(sizeof(float) * WARPS * ROWS * (HD + 4) <= SMEM, "the warps' outputs take the tiles' place");
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (blockIdx.x == 0) packed_check(a, tid, WARPS * 32);
    const int slot = blockIdx.x / a.Hkv, kh = blockIdx.x - slot * a.Hkv;
    int first;
    const int s = find_slot(a.cu_k, a.n_seq, a.total_k, A.keys, slot, first);
    if (s < 0) return;
    const int part = slot - first;
    PackedSeq p = packed_seq(a, s);
    if (a.max_k <= A.keys) p.lk = min(p.lk, A.keys);  // (reported: there is no scratch for more parts)
    const int lq = min(p.lq, A.rows / A.group), R = lq * A.group;
    const int k0 = part * A.keys, k1 = min(p.lk, k0 + A.keys);
    if (lq == 0 || (part && k0 >= p.lk)) return;

    const int n = lane / 4, t = lane % 4;
    // Q of rows n and n + 8
    uint32_t q[4][4];
    int vis[2];  // keys that the row sees
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int r = n + 8 * h, i = r / A.group;
        vis[h] = r < R ? i + 1 + p.lk - p.lq : 0;
        uint4 u[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (r < R) {
            const bf16* row = (const bf16*)a.q + (int64_t)(p.q0 + i) * a.q_stride + (kh * A.group + r - i * A.group) * HD;
            u[0] = *reinterpret_cast<const uint4*>(row + t * 8);
            u[1] = *reinterpret_cast<const uint4*>(row + 32 + t * 8);
        }
#pragma unroll
        for (int e = 0; e < 2; e++) {
            q[2 * e][h] = u[e].x;
            q[2 * e][2 + h] = u[e].y;
            q[2 * e + 1][h] = u[e].z;
            q[2 * e + 1][2 + h] = u[e].w;
        }
    }
    const bf16* kb = (const bf16*)a.k + (int64_t)p.k0 * a.k_stride + kh * HD + t * 8;
    const bf16* vb = (const bf16*)a.v + (int64_t)p.k0 * a.v_stride + kh * HD + n * 8;
    uint4* mine = reinterpret_cast<uint4*>(smem + warp * NST * STAGE) + lane;  // piece i of stage b at (16 b + i) * 32
    auto copy = [&](int buf, int i, const bf16* src, int key) {
        const uint32_t dst = (uint32_t)__cvta_generic_to_shared(mine + (16 * buf + i) * 32);
        // nothing is read, and zeros come, for a key behind the part
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(key < k1 ? 16 : 0)
                     : "memory");
    };
    auto load = [&](int buf, int at) {
        if (at < k1) {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int key = at + 8 * j + n;
                const bf16* src = kb + (int64_t)min(key, k1 - 1) * a.k_stride;
                copy(buf, 2 * j, src, key);
                copy(buf, 2 * j + 1, src + 32, key);
            }
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int key = at + 16 * (j >> 2) + 2 * t + (j & 1) + 8 * ((j >> 1) & 1);
                copy(buf, 8 + j, vb + (int64_t)min(key, k1 - 1) * a.v_stride, key);
            }
        }
        cp_async_commit();
    };
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[8][4];
#pragma unroll
    for (int j = 0; j < 8; j++) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    int at = k0 + warp * TILE, buf = 0;
#pragma unroll
    for (int i = 0; i < NST - 1; i++) load(i, at + i * STEP);
    for (; at < k1; at += STEP, buf = buf == NST - 1 ? 0 : buf + 1) {
        load(buf == 0 ? NST - 1 : buf - 1, at + (NST - 1) * STEP);
        cp_async_wait<NST - 1>();
        const uint4* tile = mine + buf * 16 * 32;
        float c[4][4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const uint4 ku = tile[(2 * j + e) * 32];
                mma(c[j], q[2 * e], ku.x, ku.y);
                mma(c[j], q[2 * e + 1], ku.z, ku.w);
            }
        }
        const int seen = min(min(vis[0], vis[1]), k1);
        if (__any_sync(0xffffffffu, at + TILE > seen)) {
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (at + 8 * j + 2 * t + (e & 1) >= min(vis[e >> 1], k1)) c[j][e] = -INFINITY;
        }
#pragma unroll
        for (int h = 0; h < 2; h++) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; j++) mx = fmaxf(mx, fmaxf(c[j][2 * h], c[j][2 * h + 1]));
            const float nm = fmaxf(m[h], quad_max(mx) * A.scale_log2);
            const float f = carry(m[h], nm), ref = nm == -INFINITY ? 0.f : nm;
            m[h] = nm;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const float w = ex2_approx(fmaf(c[j][2 * h + e], A.scale_log2, -ref));
                    c[j][2 * h + e] = w;
                    sum += w;
                }
            l[h] = l[h] * f + sum;
#pragma unroll
            for (int j = 0; j < 8; j++) {
                o[j][2 * h] *= f;
                o[j][2 * h + 1] *= f;
            }
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint32_t pa[4] = {pack2(c[2 * i][0], c[2 * i][1]), pack2(c[2 * i][2], c[2 * i][3]),
                                    pack2(c[2 * i + 1][0], c[2 * i + 1][1]), pack2(c[2 * i + 1][2], c[2 * i + 1][3])};
            const uint4 v0 = tile[(8 + 4 * i) * 32], v1 = tile[(9 + 4 * i) * 32], v2 = tile[(10 + 4 * i) * 32],
                        v3 = tile[(11 + 4 * i) * 32];
            const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
            const uint32_t w2[4] = {v2.x, v2.y, v2.z, v2.w}, w3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const uint32_t sel = j & 1 ? 0x7632 : 0x5410;
                mma(o[j], pa, __byte_perm(w0[j / 2], w1[j / 2], sel), __byte_perm(w2[j / 2], w3[j / 2], sel));
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();  // every warp is done with its tiles
    // the warps' results, joined by all: thread = (row, 8 dims)
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const float sum = quad_sum(l[h]);
        if (t == 0) {
            sm[warp][n + 8 * h] = m[h];
            sl[warp][n + 8 * h] = sum;
        }
#pragma unroll
        for (int e = 0; e < 2; e++)  // dims 8 (2t + e) + j
#pragma unroll
            for (int j = 0; j < 8; j += 4)
                *reinterpret_cast<float4*>(&so[warp][n + 8 * h][8 * (2 * t + e) + j]) =
                    make_float4(o[j][2 * h + e], o[j + 1][2 * h + e], o[j + 2][2 * h + e], o[j + 3][2 * h + e]);
    }
    __syncthreads();
    for (int i = tid; i < R * 8; i += WARPS * 32) {
        const int r = i / 8, d = i % 8 * 8;
        float M = -INFINITY, L = 0.f, y[8];
#pragma unroll
        for (int w = 0; w < WARPS; w++) M = fmaxf(M, sm[w][r]);
#pragma unroll
        for (int e = 0; e < 8; e++) y[e] = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; w++) {
            const float f = carry(sm[w][r], M);
            L += f * sl[w][r];
#pragma unroll
            for (int e = 0; e < 8; e++) y[e] += f * so[w][r][d + e];
        }
        if (p.lk <= A.keys) {  // the only part
            const int j = r / A.group, h = kh * A.group + r - j * A.group;
            const bool some = j + 1 + p.lk - p.lq > 0;  // the query sees a key
            const float inv = 1.f / L;
#pragma unroll
            for (int e = 0; e < 8; e++) y[e] = some ? y[e] * inv : 0.f;
            store8((bf16*)a.o + (int64_t)(p.q0 + j) * a.o_stride + h * HD + d, y);
            if (d == 0) a.lse[(int64_t)h * a.total_q + p.q0 + j] = some ? (M + log2f(L)) * LN2 : -INFINITY;
            continue;
        }
        float* out = A.scratch + ((int64_t)blockIdx.x * A.rows + r) * PART;
#pragma unroll
        for (int e = 0; e < 8; e += 2) *reinterpret_cast<float2*>(out + d + e) = make_float2(y[e], y[e + 1]);
        if (d == 0) *reinterpret_cast<float2*>(out + HD) = make_float2(M, L);
    }
}

// Joins the parts of a row: 32 threads, two dims each.
__global__ void __launch_bounds__(128) packed_few_join_kernel(const __grid_constant__ Args A) {
    const PackedAttn& a = A.a;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are written
    const int i = blockIdx.x * 4 + threadIdx.x / 32, lane = threadIdx.x % 32;
    const int x = i / A.rows, r = i - x * A.rows;
    if (x >= a.n_seq * a.Hkv) return;
    const int s = x / a.Hkv, kh = x - s * a.Hkv;
    const PackedSeq p = packed_seq(a, s);
    const int q = r / A.group, h = kh * A.group + r - q * A.group;
    if (q >= min(p.lq, A.rows / A.group) || p.lk <= A.keys) return;
    const int parts = (p.lk + A.keys - 1) / A.keys;
    const float* in = A.scratch + ((int64_t)((p.k0 / A.keys + s) * a.Hkv + kh) * A.rows + r) * PART;
    const int64_t step = (int64_t)a.Hkv * A.rows * PART;
    float M = -INFINITY;
    for (int k = lane; k < parts; k += 32) M = fmaxf(M, in[k * step + HD]);
    M = warp_max(M);
    float L = 0.f, y0 = 0.f, y1 = 0.f;
    for (int k = 0; k < parts; k++) {
        const float2 ml = *reinterpret_cast<const float2*>(in + k * step + HD);
        const float2 v = *reinterpret_cast<const float2*>(in + k * step + 2 * lane);
        const float f = carry(ml.x, M);
        L += f * ml.y;
        y0 += f * v.x;
        y1 += f * v.y;
    }
    const bool some = q + 1 + p.lk - p.lq > 0;
    const float inv = some ? 1.f / L : 0.f;
    if (!some) y0 = y1 = 0.f;
    *reinterpret_cast<uint32_t*>((bf16*)a.o + (int64_t)(p.q0 + q) * a.o_stride + h * HD + 2 * lane) =
        pack2(y0 * inv, y1 * inv);
    if (lane == 0) a.lse[(int64_t)h * a.total_q + p.q0 + q] = some ? (M + log2f(L)) * LN2 : -INFINITY;
}

// Keys of a part: all keys make about four blocks per SM (two at a time; 64 new
// tokens over 177402 keys of 4 heads took 47 us with two to eight, 52 with one
// long part each), at least two turns of a block.
int part_keys(int n_seq, int total_k, int max_k, int Hkv) {
    const int64_t all = min((int64_t)total_k, (int64_t)n_seq * max_k) * Hkv;
    const int64_t want = all / FILL;
    const int64_t keys = (want + STEP - 1) / STEP * STEP;
    return (int)max((int64_t)2 * STEP, keys);
}

}  // namespace

bool attention_packed_few(int max_q, int Hq, int Hkv) { return (int64_t)max_q * (Hq / Hkv) <= ROWS; }

size_t attention_packed_few_scratch(int n_seq, int total_k, int max_q, int max_k, int Hq, int Hkv) {
    const int keys = part_keys(n_seq, total_k, max_k, Hkv);
    if (max_k <= keys) return 0;
    return (size_t)packed_slots(total_k, n_seq, keys) * Hkv * max_q * (Hq / Hkv) * PART * 4;
}

int launch_attention_packed_few(const PackedAttn& a, void* scratch, cudaStream_t s) {
    Args A;
    A.a = a;
    A.group = a.Hq / a.Hkv;
    A.keys = part_keys(a.n_seq, a.total_k, a.max_k, a.Hkv);
    A.rows = a.max_q * A.group;
    A.scale_log2 = LOG2E / sqrtf((float)HD);
    A.scratch = (float*)scratch;
    if (smem_attr((const void*)packed_few_kernel, SMEM) != cudaSuccess) return GPT2_ERR_CUDA;
    packed_few_kernel<<<packed_slots(a.total_k, a.n_seq, A.keys) * a.Hkv, WARPS * 32, SMEM, s>>>(A);
    if (a.max_k <= A.keys) return 1;
    const int blocks = (int)(((int64_t)a.n_seq * a.Hkv * A.rows + 3) / 4);
    return launch_dependent(packed_few_join_kernel, blocks, 128, 0, s, A) == cudaSuccess ? 2 : GPT2_ERR_CUDA;
}
