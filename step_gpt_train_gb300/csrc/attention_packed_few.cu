// Packed attention forward for few queries (bf16, head size 64): at most 16
// rows (queries x heads of a group) per sequence and key head, one new token
// each above all. Bound by reading the keys and values once from HBM, so the
// products need only keep up: mma.sync on 16 rows, straight from registers.
//
// The keys of the whole batch are one line of rows, cut into chunks of equal
// length whatever the sequences'. A block takes one chunk and goes through the
// sequences that it meets, a warp for each of (up to) four neighbouring key
// heads, so all blocks are on the SMs at once and end together: 64 new tokens
// over 177402 keys of 4 heads (182 MB) took 47 us with a block for a part of
// one sequence and one head, 39 so. A sequence inside one chunk is written at
// once; of the others each chunk leaves its part (O, m, l) in scratch, and a
// second kernel joins them (about 5 us of the 39). Where no sequence has more
// than 128 keys none is cut, which saves the second kernel: of 64 keys 4
// sequences take 6.3 us whole and 8.3 cut (1024 of 4 heads 14 and 35), of 128
// keys 8.3 and 8.3 (27 and 49), of 192 keys 9.3 and 8.3, of 512 keys 16.6 and
// 8.4. (Batches of hundreds of sequences would gain from whole ones beyond that:
// 1024 of 512 keys and 4 heads 84 and 107.)
//
// The block's warps copy whole rows of its heads to shared memory (cp.async),
// NST - 1 tiles ahead and across the ends of sequences: 512 bytes of one row to
// a warp's instruction. What an instruction reads has to be contiguous: with
// each warp copying its own head's 128 bytes of four rows the loads alone took
// 44 us, with 512 contiguous bytes 36 (12 heads of 128 bytes: 27 us to 21).
// A block of fewer heads (their number is not a multiple of four) has fewer
// warps, and more blocks fit: 64 new tokens over caches of up to 8192 keys read
// 6.8 TB/s with 24 heads, 6.3 with 25 (a warp to a block, 128 bytes at a time).
//
// The contraction's order is free as long as both sides agree, so 16 bytes are
// used as they come. Q K^T: thread (n = lane / 4, t = lane % 4) takes dims
// 8t .. 8t+7 and 32+8t .. of key n, its 32-bit words being the fragments'
// (k, k+1) pairs, and of rows n, n + 8 of Q alike. P V: it takes dims 8n ..
// 8n+7 of keys 2t, 2t+1, 2t+8, 2t+9; byte permutes pair the keys, column n of
// the j-th product being dim 8n + j. So a thread ends with 16 consecutive
// outputs of two rows.
#include "attention_packed.cuh"

namespace {

constexpr int HD = 64;
constexpr int WARPS = 4;                   // of a block at most
constexpr int TILE = 16;                   // keys
constexpr int ROWS = 16;
constexpr int NST = 3;                     // tiles that a warp has in shared memory or on their way
constexpr int STAGE = TILE * HD * 2 * 2;   // bytes of a tile for each warp
constexpr int PART = HD + 2;               // floats of a row's partial result: O, m, l
constexpr int FILL = 16 * PACKED_SMS;      // warps at work at once
constexpr int MIN_KEYS = 32;               // of a chunk: what a block has on its way at once
constexpr int WHOLE = 128;                 // longest sequence of a batch whose sequences are not cut
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
// The reference that scores are taken against may fall behind the maximum by
// this (a factor of 256) before the sums are moved to a new one.
constexpr float SLACK = 8.f;

struct Args {
    PackedAttn a;
    int group;
    int rows;    // rows of scratch per (slot, key head)
    int chunks;  // at most; 0: a block takes a whole sequence
    float scale_log2;
    float* scratch;  // [slot][key head][rows][PART]; the slot of chunk c's part of sequence s is c + s
};

// Keys of a chunk, and the chunks that hold any (one at least). (Rows stay below 2^30.)
struct Cut {
    int total, keys, chunks;
};
__device__ __forceinline__ Cut cut_of(const Args& A) {
    Cut c;
    c.total = min(max(A.a.cu_k[A.a.n_seq], 0), A.a.total_k);
    const unsigned even = ((unsigned)c.total + A.chunks - 1) / (unsigned)A.chunks;
    c.keys = max(MIN_KEYS, (int)(even + TILE - 1) / TILE * TILE);
    c.chunks = max(1, (int)(((unsigned)c.total + c.keys - 1) / (unsigned)c.keys));
    return c;
}
// The first sequence with keys at or behind a row, or that starts there, found
// by a whole warp: 32 probes a round, those of the first on their way before the row is known.
struct Search {
    int step, c0, c1;
    __device__ __forceinline__ void probe(const int32_t* cu, int lo, int hi) {
        step = (hi - lo + 31) / 32;
        const int s = lo + (threadIdx.x & 31) * step;
        c0 = s < hi ? cu[s] : INT_MAX;
        c1 = s < hi ? cu[s + 1] : 0;
    }
    __device__ __forceinline__ int find(const int32_t* cu, int n_seq, int row) {
        int lo = 0, hi = n_seq;
        while (true) {
            const int c = __popc(__ballot_sync(0xffffffffu, c0 < row && c1 <= row));
            if (c == 0) return lo;
            hi = min(hi, lo + c * step);
            lo += (c - 1) * step + 1;
            if (lo >= hi) return lo;
            probe(cu, lo, hi);
        }
    }
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
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, warps = blockDim.x / 32;
    const int blocks = a.Hkv / warps, chunk = blockIdx.x / blocks;
    const int lead = (blockIdx.x - chunk * blocks) * warps, kh = lead + warp;
    if (blockIdx.x == 0) packed_check(a, tid, blockDim.x);
    const bool whole = A.chunks == 0;
    bool final = whole;  // no chunk behind this one
    int c0, c1;
    Search search;
    if (whole) {
        const PackedSeq p = packed_seq(a, chunk);
        c0 = p.k0;
        c1 = p.k0 + p.lk;
    } else {
        search.probe(a.cu_k, 0, a.n_seq);
        const Cut cut = cut_of(A);
        if (chunk >= cut.chunks) return;
        final = chunk == cut.chunks - 1;
        c0 = chunk * cut.keys;
        c1 = min(cut.total, c0 + cut.keys);
    }

    // Copies: 16 bytes of every fourth row of the block's heads. Places: [tile][K, V][head][key][16 bytes], the last
    // index turned by the key so that eight lanes of a reading warp find eight different 16 bytes of a 128-byte line.
    const int row = tid / (8 * warps), piece = tid - row * 8 * warps;
    const bf16* kb = (const bf16*)a.k + (c0 + row) * a.k_stride + lead * HD + piece * 8;
    const bf16* vb = (const bf16*)a.v + (c0 + row) * a.v_stride + lead * HD + piece * 8;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem), half = warps * TILE * HD * 2;
    const uint32_t to = base + (piece / 8 * TILE + row) * 128;
    const uint32_t k_at = to + ((piece ^ (row & 1) << 2) & 7) * 16;                  // rows row + 4 j
    const uint32_t v_at = to + half + ((piece ^ (row & 2)) & 7) * 16;                // j even; odd: ^ 64
    auto copy = [&](uint32_t to, const bf16* src, int bytes) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(bytes) : "memory");
    };
    auto fetch = [&](int i) {  // tile i of the chunk
        const int left = c1 - c0 - i * TILE;
        const uint32_t buf = i % NST * 2 * half;
        const bf16* k = kb + i * TILE * a.k_stride;
        const bf16* v = vb + i * TILE * a.v_stride;
        if (left >= TILE) {
#pragma unroll
            for (int j = 0; j < TILE / 4; j++) copy(k_at + buf + j * 512, k + 4 * j * a.k_stride, 16);
#pragma unroll
            for (int j = 0; j < TILE / 4; j++) copy((v_at ^ (j & 1) * 64) + buf + j * 512, v + 4 * j * a.v_stride, 16);
        } else if (left > 0) {  // nothing is read, and zeros come, for a row behind the chunk
#pragma unroll
            for (int j = 0; j < TILE / 4; j++) {
                const bool in = row + 4 * j < left;
                copy(k_at + buf + j * 512, in ? k + 4 * j * a.k_stride : (const bf16*)a.k, in ? 16 : 0);
                copy((v_at ^ (j & 1) * 64) + buf + j * 512, in ? v + 4 * j * a.v_stride : (const bf16*)a.v, in ? 16 : 0);
            }
        }
        cp_async_commit();
    };
    int ready = -1, ahead = 0;  // the last tile that is there for all warps; the first that is not on its way
    for (; ahead < NST - 1; ahead++) fetch(ahead);
    // (all warps of the block go through the same tiles)
    auto arrive = [&](int i) {
        while (ready < i) {
            cp_async_wait<NST - 2>();
            __syncthreads();  // tile ready + 1 is there, and nobody reads the place of the one before any more
            ready++;
            fetch(ahead++);
        }
    };
    const int n = lane / 4, t = lane % 4;
    const uint8_t* kt = smem + (warp * TILE + n) * 128 + (t ^ (n & 1) << 2) * 16;
    const uint8_t* vt = smem + half + (warp * TILE + 2 * t) * 128 + (n ^ t << 1) * 16;

    const int end = whole ? chunk + 1 : a.n_seq;
    for (int s = whole ? chunk : search.find(a.cu_k, a.n_seq, c0); s < end; s++) {
        const PackedSeq p = packed_seq(a, s);
        if (p.k0 >= c1 && !final) break;
        const int lq = min(p.lq, A.rows / A.group), R = lq * A.group;
        const int a0 = max(p.k0, c0), a1 = min(p.k0 + p.lk, c1);  // the chunk's rows of the sequence
        if (lq == 0 || (a0 >= a1 && p.lk)) continue;
        int i = (a0 - c0) / TILE;
        if (i >= ahead) {  // tiles that nothing asks for are skipped
            cp_async_wait<0>();
            __syncthreads();
            ready = i - 1;
            for (ahead = i; ahead < i + NST - 1; ahead++) fetch(ahead);
        }
        // Q of rows n and n + 8
        uint32_t q[4][4];
        int sees[2];  // the row sees the buffer's keys before this one (rows that are not there: zeros, nothing masked)
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int r = n + 8 * h, j = r / A.group;
            sees[h] = p.k0 + p.lk + (r < R ? j + 1 - p.lq : 0);
            uint4 u[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            if (r < R) {
                const bf16* row = (const bf16*)a.q + (p.q0 + j) * a.q_stride + (kh * A.group + r - j * A.group) * HD;
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
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[8][4];
#pragma unroll
        for (int j = 0; j < 8; j++) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        for (; c0 + i * TILE < a1; i++) {
            arrive(i);
            const uint32_t buf = i % NST * 2 * half;
            const int at = c0 + i * TILE;
            float c[TILE / 8][4];
#pragma unroll
            for (int j = 0; j < TILE / 8; j++) {
                c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.f;
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const uint4 ku = *reinterpret_cast<const uint4*>(kt + buf + j * 1024 + (e ? (n & 1 ? -64 : 64) : 0));
                    mma(c[j], q[2 * e], ku.x, ku.y);
                    mma(c[j], q[2 * e + 1], ku.z, ku.w);
                }
            }
            const bool edge = at < a0 || at + TILE > a1;  // the tile has other sequences' rows, or none
            if (edge || __any_sync(0xffffffffu, at + TILE > min(sees[0], sees[1]))) {
#pragma unroll
                for (int j = 0; j < TILE / 8; j++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int key = at + 8 * j + 2 * t + (e & 1);
                        if (key < a0 || key >= min(sees[e >> 1], a1)) c[j][e] = -INFINITY;
                    }
            }
            float top[2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                top[h] = -INFINITY;
#pragma unroll
                for (int j = 0; j < TILE / 8; j++) top[h] = fmaxf(top[h], fmaxf(c[j][2 * h], c[j][2 * h + 1]));
                top[h] *= A.scale_log2;
            }
            if (__any_sync(0xffffffffu, top[0] > m[0] + SLACK || top[1] > m[1] + SLACK)) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float nm = fmaxf(m[h], quad_max(top[h])), f = carry(m[h], nm);
                    m[h] = nm;
                    l[h] *= f;
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        o[j][2 * h] *= f;
                        o[j][2 * h + 1] *= f;
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const float ref = m[h] == -INFINITY ? 0.f : -m[h];
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < TILE / 8; j++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const float x = ex2_approx(fmaf(c[j][2 * h + e], A.scale_log2, ref));
                        c[j][2 * h + e] = x;
                        sum += x;
                    }
                l[h] += sum;
            }
#pragma unroll
            for (int b = 0; b < TILE / 16; b++) {
                const uint32_t pa[4] = {pack2(c[2 * b][0], c[2 * b][1]), pack2(c[2 * b][2], c[2 * b][3]),
                                        pack2(c[2 * b + 1][0], c[2 * b + 1][1]), pack2(c[2 * b + 1][2], c[2 * b + 1][3])};
                uint4 v[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    v[j] = *reinterpret_cast<const uint4*>(vt + buf + (16 * b + (j & 1) + 8 * (j >> 1)) * 128);
                    const int key = at + 16 * b + 2 * t + (j & 1) + 8 * (j >> 1);
                    if (edge && (key < a0 || key >= a1)) v[j] = make_uint4(0, 0, 0, 0);  // 0 x another's NaN
                }
                const uint32_t v0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, v1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
                const uint32_t v2[4] = {v[2].x, v[2].y, v[2].z, v[2].w}, v3[4] = {v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const uint32_t sel = j & 1 ? 0x7632 : 0x5410;
                    mma(o[j], pa, __byte_perm(v0[j / 2], v1[j / 2], sel), __byte_perm(v2[j / 2], v3[j / 2], sel));
                }
            }
            if (at + TILE > a1) break;  // the next sequence begins in this tile
        }
        // thread: rows n, n + 8, dims 16t .. 16t + 15
        const bool all = a1 - a0 == p.lk || A.chunks <= 1;  // the whole sequence
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int r = n + 8 * h, j = r / A.group, head = kh * A.group + r - j * A.group;
            const float sum = quad_sum(l[h]);
            if (r >= R) continue;
            if (all) {
                const bool some = sees[h] > p.k0;  // the query sees a key
                const float inv = some ? 1.f / sum : 0.f;
                bf16* out = (bf16*)a.o + (p.q0 + j) * a.o_stride + head * HD + 16 * t;
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float y[8];
#pragma unroll
                    for (int d = 0; d < 8; d++) y[d] = some ? o[d][2 * h + e] * inv : 0.f;
                    store8(out + 8 * e, y);
                }
                if (t == 0) a.lse[(int64_t)head * a.total_q + p.q0 + j] = some ? (m[h] + log2f(sum)) * LN2 : -INFINITY;
            } else {
                float* out = A.scratch + ((((int64_t)chunk + s) * a.Hkv + kh) * A.rows + r) * PART;
#pragma unroll
                for (int e = 0; e < 2; e++)
#pragma unroll
                    for (int d = 0; d < 8; d += 2)
                        *reinterpret_cast<float2*>(out + 16 * t + 8 * e + d) =
                            make_float2(o[d][2 * h + e], o[d + 1][2 * h + e]);
                if (t == 0) *reinterpret_cast<float2*>(out + HD) = make_float2(m[h], sum);
            }
        }
    }
    cp_async_wait<0>();
}

// Joins the parts of a row: four warps take them in turn, AT_ONCE on their way to each, a lane two dims.
constexpr int AT_ONCE = 4;
__global__ void __launch_bounds__(128) packed_few_join_kernel(const __grid_constant__ Args A) {
    const PackedAttn& a = A.a;
    __shared__ float sm[4], sl[4], so[4][HD];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int x = blockIdx.x / A.rows, r = blockIdx.x - x * A.rows;
    const int s = x / a.Hkv, kh = x - s * a.Hkv;
    const PackedSeq p = packed_seq(a, s);
    const Cut cut = cut_of(A);
    const int q = r / A.group, h = kh * A.group + r - q * A.group;
    const int first = min(p.k0 / cut.keys, cut.chunks - 1);
    const int parts = min((p.k0 + p.lk - 1) / cut.keys, cut.chunks - 1) - first + 1;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are written
    if (q >= min(p.lq, A.rows / A.group) || p.lk == 0 || parts <= 1) return;
    const float* in = A.scratch + ((((int64_t)first + s) * a.Hkv + kh) * A.rows + r) * PART;
    const int64_t step = (int64_t)a.Hkv * A.rows * PART;
    float M = -INFINITY, L = 0.f, y0 = 0.f, y1 = 0.f;
    for (int k = warp; k < parts; k += 4 * AT_ONCE) {
        float2 ml[AT_ONCE], v[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; i++) {
            const bool in_range = k + 4 * i < parts;
            const float* x = in + (in_range ? k + 4 * i : k) * step;
            ml[i] = *reinterpret_cast<const float2*>(x + HD);
            v[i] = *reinterpret_cast<const float2*>(x + 2 * lane);
            if (!in_range) ml[i] = make_float2(-INFINITY, 0.f);
        }
        float top = M;
#pragma unroll
        for (int i = 0; i < AT_ONCE; i++) top = fmaxf(top, ml[i].x);
        const float f = carry(M, top);
        L *= f, y0 *= f, y1 *= f, M = top;
#pragma unroll
        for (int i = 0; i < AT_ONCE; i++) {
            const float f = carry(ml[i].x, M);
            if (k + 4 * i >= parts) break;
            L += f * ml[i].y;
            y0 += f * v[i].x;
            y1 += f * v[i].y;
        }
    }
    if (lane == 0) sm[warp] = M, sl[warp] = L;
    *reinterpret_cast<float2*>(&so[warp][2 * lane]) = make_float2(y0, y1);
    __syncthreads();
    if (warp) return;
    const bool some = q + 1 + p.lk - p.lq > 0;
    M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    L = y0 = y1 = 0.f;
    for (int k = 0; k < 4; k++) {
        const float f = carry(sm[k], M);
        L += f * sl[k];
        y0 += f * so[k][2 * lane];
        y1 += f * so[k][2 * lane + 1];
    }
    const float inv = some ? 1.f / L : 0.f;
    if (!some) y0 = y1 = 0.f;
    *reinterpret_cast<uint32_t*>((bf16*)a.o + (p.q0 + q) * a.o_stride + h * HD + 2 * lane) = pack2(y0 * inv, y1 * inv);
    if (lane == 0) a.lse[(int64_t)h * a.total_q + p.q0 + q] = some ? (M + log2f(L)) * LN2 : -INFINITY;
}

int chunks_of(int n_seq, int total_k, int max_k, int Hkv) {
    if (max_k <= WHOLE) return 0;
    const int64_t all = min((int64_t)total_k, (int64_t)n_seq * max_k);
    return (int)max((int64_t)1, min((int64_t)FILL / Hkv, (all + MIN_KEYS - 1) / MIN_KEYS));
}

}  // namespace

bool attention_packed_few(int max_q, int Hq, int Hkv) { return (int64_t)max_q * (Hq / Hkv) <= ROWS; }

size_t attention_packed_few_scratch(int n_seq, int total_k, int max_q, int max_k, int Hq, int Hkv) {
    const int chunks = chunks_of(n_seq, total_k, max_k, Hkv);
    if (chunks <= 1) return 0;
    return (size_t)(chunks + n_seq) * Hkv * max_q * (Hq / Hkv) * PART * 4;
}

int launch_attention_packed_few(const PackedAttn& a, void* scratch, cudaStream_t s) {
    Args A;
    A.a = a;
    A.group = a.Hq / a.Hkv;
    A.rows = a.max_q * A.group;
    A.chunks = chunks_of(a.n_seq, a.total_k, a.max_k, a.Hkv);
    A.scale_log2 = LOG2E / sqrtf((float)HD);
    A.scratch = (float*)scratch;
    int warps = WARPS;
    while (a.Hkv % warps) warps /= 2;
    if (smem_attr((const void*)packed_few_kernel, WARPS * NST * STAGE) != cudaSuccess) return GPT2_ERR_CUDA;
    packed_few_kernel<<<(A.chunks ? A.chunks : a.n_seq) * (a.Hkv / warps), warps * 32, warps * NST * STAGE, s>>>(A);
    if (A.chunks <= 1 || A.rows == 0) return 1;
    return launch_dependent(packed_few_join_kernel, a.n_seq * a.Hkv * A.rows, 128, 0, s, A) == cudaSuccess
               ? 2
               : GPT2_ERR_CUDA;
}
