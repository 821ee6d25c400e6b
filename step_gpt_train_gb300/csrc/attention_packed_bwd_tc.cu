// Packed causal attention backward on the tcgen05 tensor cores (bf16, head
// size 64, grouped heads up to 64): two deterministic kernels of one template,
// no atomics, one writer for every gradient.
//
//   dK, dV: an item is a tile of 128 keys of one key head; it walks the blocks
//     of 64 rows (queries x the group's heads, in this order, as the forward
//     lays them out) that see it, so the sum over shared heads is part of the
//     products' long dimension:
//       S^T = K Q^T, dP^T = V dO^T                  (M=128 keys, N=64 rows, K=64)
//       P^T = exp2(S^T log2(e)/sqrt(hd) - lse log2(e)), dS^T = P^T (dP^T - D)
//       dV += P^T dO, dK += dS^T Q                  (M=128, N=64, K=64)
//   dQ: an item is a tile of 128 rows; it walks blocks of 64 keys:
//       S = Q K^T, dP = dO V^T, dS as above, dQ += dS K.
//
// So both are a resident pair of tiles A1, A2 (double-buffered across items),
// a ring of streamed pairs B1, B2, and S = A1 B1^T, dP = A2 B2^T, acc1 += P B2
// (dK, dV only), acc0 += dS B1, with P and dS going back to TMEM as bf16 pairs
// (their one rounding), the products' A operand.
//
// A step's chain (wait, load S, exponentials, store P, wait, load dP, store dS)
// is all latency, so two steps are in flight: even and odd steps have their own
// TMEM buffers (S, dP, P, dS: 192 columns each) and their own eight elementwise
// warps (32 columns a thread). One warp issues all accumulations, in step order,
// which fixes the order of every sum; another S and dP, two steps ahead.
//
// Warps: 0 TMA producer; 1, 3 MMA; 2 work items (ring of two), rows of a block
// behind the sequence's end set to zero (0 * NaN from a neighbour would reach
// the accumulators), outputs of items that meet nothing; 4..7 accumulators out
// (while the next item runs); 8..15, 16..23 elementwise. Every wait is bounded.
// Before them a pass forms D = rowsum(dO * O) and lse log2(e) per row and sorts
// the items.
//
// Measured: 62 documents of 100 to 1024 tokens, 12 heads, 174 us in all (50
// GFLOP: 285 TFLOP/s; HBM would take 44). Bound by the elementwise warps' chain;
// the tensor cores are busy 22% of the time in either kernel.
#include "attention_packed_tc.cuh"

namespace {

using namespace packed_tc;

constexpr int BLK = 64;             // rows or keys of a streamed block
constexpr int BT = BLK * HD * 2;    // 8 KB
constexpr int NB = 4;               // streamed stages
constexpr int NIT = 2;              // work item ring: an item is drawn when the one before it begins, not earlier
constexpr int EW = 8;               // elementwise warps of a step
constexpr int THREADS = 32 * (8 + 2 * EW);
// TMEM columns: step parity p at 192 p: S, dP (fp32), P, dS (bf16 pairs); accumulators
constexpr uint32_t T_S = 0, T_DP = 64, T_P = 128, T_DS = 160, T_STEP = 192, T_ACC0 = 384, T_ACC1 = 448;
// shared memory: A1, A2 [2 items] | B1, B2 [NB] | staging per output warp | per elementwise warp 64 floats | items | barriers
constexpr int OFF_B = 4 * TILE, OFF_STG = OFF_B + NB * 2 * BT, STG = 32 * 128;
constexpr int OFF_SLOT = OFF_STG + 4 * STG, OFF_IT = OFF_SLOT + 2 * EW * 256, OFF_BAR = OFF_IT + NIT * 64;
constexpr int SMEM = OFF_BAR + 512 + 1024;
static_assert(SMEM <= 232448, "shared memory per CTA");

struct Item {
    int valid, kh;       // key head
    int r0, n;           // first row (dQ: query, dK/dV: key) of the buffer, rows of the tile
    int s0, len, shift;  // the other kind: first row of the buffer, length, see PackedTile
    int first;           // dK/dV: the first query of block 0
    int nb, base;        // blocks; step counter before the item
};
static_assert(sizeof(Item) <= 64, "item slot");

struct Args {
    PackedAttn a;
    PackedAttnGrad g;
    const float2* ld;    // [Hq, total_q]: lse log2(e), D
    int group;
    int bq;              // dK/dV: queries of a block (64 / group); dQ: keys of a block (64)
    int items;
    float scale, scale_log2;
    PackedCut cut;
    PackedPlan* plan;
};

// The launches of a call overlap: the sort lets the pass that forms D start at
// once; dQ sets itself up during that pass and waits for it (which has waited
// for the sort); dK, dV starts on the SMs that dQ leaves, since it needs
// nothing from it, and ends after it.
__device__ __forceinline__ void depend_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void depend_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct PlanArgs {
    PackedAttn a;
    PackedCut cut[2];
    PackedPlan* plan[2];
};
__global__ void __launch_bounds__(1024) packed_plans_kernel(const __grid_constant__ PlanArgs A) {
    depend_launch();
    packed_plan_block(A.a, A.cut[blockIdx.x], A.plan[blockIdx.x], blockIdx.x == 0);
}

// lse log2(e) and D of every (row, head): eight lanes to each, 16 bytes of O
// and dO a lane, four pairs in flight.
constexpr int PREP = 128;  // pairs of a block
__global__ void __launch_bounds__(256) packed_prep_kernel(PackedAttn a, PackedAttnGrad g, float2* ld) {
    depend_launch();
    const int first = blockIdx.x * PREP + threadIdx.x / 8, e = threadIdx.x % 8;
    uint4 x[4], y[4];
    int64_t at[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const int i = first + k * 32;
        const bool in = i < a.total_q * a.Hq;
        const int row = in ? i / a.Hq : 0, h = in ? i - row * a.Hq : 0;
        at[k] = in ? (int64_t)h * a.total_q + row : -1;
        x[k] = __ldcs(reinterpret_cast<const uint4*>((const bf16*)a.o + (int64_t)row * a.o_stride + h * HD + e * 8));
        y[k] = *reinterpret_cast<const uint4*>((const bf16*)g.dout + (int64_t)row * g.dout_stride + h * HD + e * 8);
    }
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const uint32_t u[4] = {x[k].x, x[k].y, x[k].z, x[k].w}, v[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
        float d = 0.f;
#pragma unroll
        for (int j = 0; j < 4; j++)
            d += __uint_as_float(u[j] << 16) * __uint_as_float(v[j] << 16) +
                 __uint_as_float(u[j] & 0xFFFF0000u) * __uint_as_float(v[j] & 0xFFFF0000u);
#pragma unroll
        for (int o = 4; o > 0; o /= 2) d += __shfl_xor_sync(0xffffffffu, d, o);
        if (at[k] >= 0 && e == 0) {
            const float l = a.lse[at[k]];
            ld[at[k]] = make_float2(l == -INFINITY ? 0.f : l * LOG2E, d);
        }
    }
    depend_wait();  // the sort too is done when this pass is
}

template <bool DQ>
__global__ void __launch_bounds__(THREADS, 1)
    packed_bwd_tc_kernel(const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_a2,
                         const __grid_constant__ CUtensorMap tm_b1, const __grid_constant__ CUtensorMap tm_b2,
                         const __grid_constant__ Args A) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const PackedAttn& a = A.a;
    auto sA = [&](int buf, int k) { return base + (2 * buf + k) * TILE; };
    auto sB = [&](int st, int k) { return base + OFF_B + (2 * st + k) * BT; };
    const uint32_t bars = base + OFF_BAR;
    int nbar = 0;
    auto bar = [&](int n) { const uint32_t b = bars + 8u * nbar; nbar += n; return b; };
    const uint32_t it_full = bar(NIT), it_empty = bar(NIT), a_full = bar(2), a_empty = bar(2);
    const uint32_t b_full = bar(NB), b_empty = bar(NB), b_raw = bar(NB);
    const uint32_t s_full = bar(2), dp_full = bar(2), p_full = bar(2);
    const uint32_t ds_full = bar(2), ds_free = bar(2), acc_full = bar(2), acc_empty = bar(2), drain = bar(2);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + OFF_BAR + 496);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + OFF_BAR + 500);
    Item* ring = reinterpret_cast<Item*>(gbase + OFF_IT);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    int* status = a.status;
    const int used = DQ ? BLK : A.bq * A.group;  // rows that a block's load fills

    if (threadIdx.x == 0) {
        for (int i = 0; i < NIT; i++) {
            mbar_init(it_full + 8 * i, 1);
            mbar_init(it_empty + 8 * i, 3 + 4 + 2 * EW);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(a_full + 8 * i, 1);
            mbar_init(a_empty + 8 * i, 1);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(dp_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, EW);
            mbar_init(ds_full + 8 * i, EW);
            mbar_init(ds_free + 8 * i, 1);
        }
        for (int i = 0; i < NB; i++) {
            mbar_init(b_full + 8 * i, 1);
            mbar_init(b_empty + 8 * i, 1);
            mbar_init(b_raw + 8 * i, 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, 4);
        }
        mbar_init(drain, 1);
        mbar_init(drain + 8, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (!DQ && used < BLK) {  // rows that no load fills
        for (int i = threadIdx.x; i < NB * 2 * (BLK - used) * 8; i += THREADS) {
            const int per = max(1, BLK - used) * 8, t = i / per, e = i - t * per;
            reinterpret_cast<uint4*>(gbase + OFF_B + t * BT + used * 128)[e] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
    }
    if (warp == 1) tmem_alloc(smem_addr((const void*)tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    auto take = [&](int i, Item& it) -> bool {
        const int sl = i % NIT;
        if (!wait(it_full + 8 * sl, (i / NIT) & 1, abort_flag, status)) return false;
        it = ring[sl];
        __syncwarp();
        if (lane == 0) mbar_arrive(it_empty + 8 * sl);
        return it.valid;
    };
    // rows of block n (queries or keys) that belong to the sequence
    auto real = [&](const Item& it, int n) { return min(A.bq, it.len - it.first - n * A.bq); };

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        int a_issued[2] = {-1, -1}, b_issued[NB], r_uses[NB];
        for (int i = 0; i < NB; i++) b_issued[i] = -1, r_uses[i] = 0;
        const uint32_t a_bytes = DQ ? 2u * (128 / A.group) * A.group * HD * 2 : 2u * TILE;
        Item it;
        bool ok = true;
        for (int i = 0; ok && take(i, it); i++) {
            if (lane == 0) {
                const int buf = i & 1;
                const uint32_t ph = (uint32_t)(i >> 1) & 1u;
                ok = mbar_wait(a_empty + 8 * buf, ph ^ 1u, abort_flag, status);
                if (ok) {
                    const int h = DQ ? it.kh * A.group : it.kh;
                    mbar_expect_tx(a_full + 8 * buf, a_bytes);
                    tma_load_3d(sA(buf, 0), &tm_a1, a_full + 8 * buf, 0, h, it.r0);
                    tma_load_3d(sA(buf, 1), &tm_a2, a_full + 8 * buf, 0, h, it.r0);
                    a_issued[buf] = (int)ph;
                }
                for (int n = 0; ok && n < it.nb; n++) {
                    const int g = it.base + n, st = g % NB;
                    const uint32_t bph = (uint32_t)(g / NB) & 1u;
                    if (!(ok = mbar_wait(b_empty + 8 * st, bph ^ 1u, abort_flag, status))) break;
                    const bool tail = real(it, n) < A.bq;  // by way of the warp that zeroes the rest
                    const uint32_t bb = (tail ? b_raw : b_full) + 8 * st;
                    const int h = DQ ? it.kh : it.kh * A.group, row = it.s0 + it.first + n * A.bq;
                    mbar_expect_tx(bb, 2u * used * HD * 2);
                    tma_load_3d(sB(st, 0), &tm_b1, bb, 0, h, row);
                    tma_load_3d(sB(st, 1), &tm_b2, bb, 0, h, row);
                    r_uses[st] += tail;
                    b_issued[st] = tail ? -1 : (int)bph;  // the stage's earlier loads have been read
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        if (lane == 0) {
            for (int b = 0; b < 2; b++)
                if (a_issued[b] >= 0) mbar_drain(a_full + 8 * b, (uint32_t)a_issued[b], status);
            for (int st = 0; st < NB; st++) {
                if (b_issued[st] >= 0) mbar_drain(b_full + 8 * st, (uint32_t)b_issued[st], status);
                if (r_uses[st]) mbar_drain(b_raw + 8 * st, (uint32_t)(r_uses[st] - 1) & 1u, status);
            }
        }
        __syncwarp();
    } else if (warp == 1 || warp == 3) {
        // ------------------------------------------------------ MMA: warp 1 S and dP, warp 3 the accumulations; the
        // whole warp runs the schedule, one elected lane issues (an issue takes about 60 cycles, more than these
        // products, and a wait that passes at once 90: one warp for both took 1500 a step)
        const bool leader = elect_one();
        constexpr uint32_t idesc_s = make_idesc(128, BLK, false, false);  // K-major x K-major
        constexpr uint32_t idesc_o = make_idesc(128, HD, false, true);    // K-major x MN-major
        Item it;
        bool ok = true;
        for (int i = 0; ok && take(i, it); i++) {
            if (warp == 1) {
                if (!(ok = wait(a_full + 8 * (i & 1), (i >> 1) & 1, abort_flag, status))) break;
                const uint64_t da1 = sw128_desc(sA(i & 1, 0), 16, 1024), da2 = sw128_desc(sA(i & 1, 1), 16, 1024);
#pragma unroll 1
                for (int n = 0; n < it.nb; n++) {
                    const int g = it.base + n, st = g % NB, p = g & 1;
                    const uint32_t before = ((g >> 1) & 1) ^ 1;
                    const uint64_t db1 = sw128_desc(sB(st, 0), 16, 1024), db2 = sw128_desc(sB(st, 1), 16, 1024);
                    if (!(ok = wait(b_full + 8 * st, (g / NB) & 1, abort_flag, status))) break;
                    // S and dP go where those of step g - 2 were: free once its P (dQ: dS) and dS have come
                    if (!(ok = wait((DQ ? ds_full : p_full) + 8 * p, before, abort_flag, status))) break;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < HD / 16; k++)
                            tc_mma(tmem + T_STEP * p + T_S, da1 + 2 * k, db1 + 2 * k, idesc_s, k > 0 ? 1u : 0u);
                        tc_commit(s_full + 8 * p);
                    }
                    __syncwarp();
                    if (!DQ && !(ok = wait(ds_full + 8 * p, before, abort_flag, status))) break;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < HD / 16; k++)
                            tc_mma(tmem + T_STEP * p + T_DP, da2 + 2 * k, db2 + 2 * k, idesc_s, k > 0 ? 1u : 0u);
                        tc_commit(dp_full + 8 * p);
                        if (n == it.nb - 1) tc_commit(a_empty + 8 * (i & 1));  // the item's last read of A1, A2
                    }
                    __syncwarp();
                }
            } else {
                // dQ has the accumulators of two items, dK and dV those of one
                const int b = DQ ? i & 1 : 0;
                const uint32_t acc0 = tmem + (b ? T_ACC1 : T_ACC0);
                if (!(ok = wait(acc_empty + 8 * b, ((DQ ? i >> 1 : i) & 1) ^ 1u, abort_flag, status))) break;
#pragma unroll 1
                for (int n = 0; n < it.nb; n++) {
                    const int g = it.base + n, st = g % NB, p = g & 1;
                    const uint32_t ph = (g >> 1) & 1;
                    // MN-major B: one 16-row k step = 2048 bytes = 128 units of the address field
                    const uint64_t db1 = sw128_desc(sB(st, 0), 8192, 1024), db2 = sw128_desc(sB(st, 1), 8192, 1024);
                    if (!(ok = wait(b_full + 8 * st, (g / NB) & 1, abort_flag, status))) break;
                    if (!DQ) {
                        if (!(ok = wait(p_full + 8 * p, ph, abort_flag, status))) break;
                        tc_fence_after();
                        if (leader) {
#pragma unroll
                            for (int k = 0; k < BLK / 16; k++)
                                tc_mma_ts(tmem + T_ACC1, tmem + T_STEP * p + T_P + 8 * k, db2 + 128 * k, idesc_o,
                                          (n > 0 || k > 0) ? 1u : 0u);
                        }
                        __syncwarp();
                    }
                    if (!(ok = wait(ds_full + 8 * p, ph, abort_flag, status))) break;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < BLK / 16; k++)
                            tc_mma_ts(acc0, tmem + T_STEP * p + T_DS + 8 * k, db1 + 128 * k, idesc_o,
                                      (n > 0 || k > 0) ? 1u : 0u);
                        tc_commit(ds_free + 8 * p);
                        tc_commit(b_empty + 8 * st);
                        if (n == it.nb - 1) tc_commit(acc_full + 8 * b);
                    }
                    __syncwarp();
                }
            }
        }
        if (leader) tc_commit(drain + 8 * (warp >> 1));
        mbar_drain(drain + 8 * (warp >> 1), 0, status);
    } else if (warp == 2) {
        // ------------------------------------------------------ work items, tails of blocks
        int x = blockIdx.x, steps = 0;
        if (DQ) {
            depend_wait();    // the sort and D are there
            depend_launch();  // dK, dV may start where this kernel has ended
        }
        if (DQ && blockIdx.x == 0 && !A.plan) packed_check(a, lane, 32);
        auto put = [&](int i, Item& it) -> bool {  // the next item, or the end, into ring slot i
            PackedTile p;
            while ((it.valid = next_tile(a, A.cut, A.plan, A.items, x, p, it.kh)) != 0) {
                it.nb = A.cut.blocks(p, p.n);
                if (it.nb) break;
                // meets nothing: its gradients are 0
                const int per = DQ ? A.group * 8 : 8;  // 16-byte units of a row
                for (int e = lane; e < p.n * per; e += 32) {
                    const int r = e / per, u = e - r * per;
                    const int64_t row = p.r0 + r;
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    if (DQ) {
                        *reinterpret_cast<uint4*>((bf16*)A.g.dq + row * A.g.dq_stride + it.kh * A.group * HD + u * 8) = zero;
                    } else {
                        *reinterpret_cast<uint4*>((bf16*)A.g.dk + row * A.g.dk_stride + it.kh * HD + u * 8) = zero;
                        *reinterpret_cast<uint4*>((bf16*)A.g.dv + row * A.g.dv_stride + it.kh * HD + u * 8) = zero;
                    }
                }
            }
            if (it.valid) {
                it.r0 = p.r0;
                it.n = p.n;
                it.s0 = p.s0;
                it.len = p.len;
                it.shift = p.shift;
                it.first = A.cut.first(p);
                it.base = steps;
                steps += it.nb;
            }
            const int sl = i % NIT;
            if (!wait(it_empty + 8 * sl, ((i / NIT) & 1) ^ 1u, abort_flag, status)) return false;
            if (lane == 0) {
                ring[sl] = it;
                mbar_arrive(it_full + 8 * sl);
            }
            __syncwarp();
            return true;
        };
        int uses[NB];
        for (int i = 0; i < NB; i++) uses[i] = 0;
        Item cur, nxt;
        bool ok = put(0, cur);
#pragma unroll 1
        for (int i = 0; ok && cur.valid; i++) {
            ok = put(i + 1, nxt);
            const int n = cur.nb - 1, left = real(cur, n);
            if (ok && left < A.bq) {
                const int st = (cur.base + n) % NB;
                int u = 0;
#pragma unroll
                for (int e = 0; e < NB; e++)
                    if (e == st) u = uses[e]++;
                if (!(ok = wait(b_raw + 8 * st, u & 1, abort_flag, status))) break;
                const int from = DQ ? left : left * A.group;
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    uint4* t = reinterpret_cast<uint4*>(gbase + OFF_B + (2 * st + k) * BT);
                    for (int e = from * 8 + lane; e < BLK * 8; e += 32) t[e] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_full + 8 * st);
            }
            cur = nxt;
        }
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------------ accumulators out
        const int quad = warp & 3, r = quad * 32 + lane;  // row of the tile = TMEM lane
        const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
        uint8_t* st = gbase + OFF_STG + quad * STG;
        uint8_t* my = st + lane * 128;
        const int qi = DQ ? r / A.group : r, hg = DQ ? r - qi * A.group : 0;
        Item it;
        bool ok = true;
#pragma unroll 1
        for (int i = 0; ok && take(i, it); i++) {
            const int b = DQ ? i & 1 : 0;
            if (!(ok = wait(acc_full + 8 * b, (DQ ? i >> 1 : i) & 1, abort_flag, status))) break;
            tc_fence_after();
            const bool mine = qi < it.n;  // (dQ: a tile's unused last rows lie behind its n queries)
#pragma unroll 1
            for (int k = DQ ? 0 : 1; k >= 0; k--) {  // dV, dK or dQ alone
                const float s = k ? 1.f : A.scale;
#pragma unroll
                for (int hh = 0; hh < 2; hh++) {
                    uint32_t v[32];
                    tc_ld32_issue(trow + (k || b ? T_ACC1 : T_ACC0) + 32 * hh, v);
                    tc_ld_wait(v);
                    if (k == 0 && hh == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(acc_empty + 8 * b);
                    }
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        uint32_t w[4];
#pragma unroll
                        for (int u = 0; u < 4; u++)
                            w[u] = cvt_bf16x2(__uint_as_float(v[c * 8 + 2 * u]) * s,
                                              __uint_as_float(v[c * 8 + 2 * u + 1]) * s);
                        *reinterpret_cast<uint4*>(my + (((hh * 4 + c) ^ (lane & 7)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                bf16* o = reinterpret_cast<bf16*>(DQ ? A.g.dq : k ? A.g.dv : A.g.dk);
                const int64_t stride = DQ ? A.g.dq_stride : k ? A.g.dv_stride : A.g.dk_stride;
                const int64_t off = mine ? (it.r0 + qi) * stride + ((DQ ? it.kh * A.group : it.kh) + hg) * HD : -1;
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int sr = e * 4 + (lane >> 3), c = lane & 7;
                    const int64_t at = __shfl_sync(0xffffffffu, off, sr);
                    const uint4 w = *reinterpret_cast<const uint4*>(st + sr * 128 + ((c ^ (sr & 7)) << 4));
                    if (at >= 0) *reinterpret_cast<uint4*>(o + at + c * 8) = w;
                }
                __syncwarp();  // the staged rows have been read
            }
        }
    } else if (warp >= 8) {
        // ------------------------------------------------------ elementwise, steps of parity `odd`
        const int ew = warp - 8, odd = ew / EW, half = (ew >> 2) & 1, quad = warp & 3;
        const int r = quad * 32 + lane;  // row of the tile = TMEM lane
        const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16) + T_STEP * odd;
        const uint32_t tS = trow + T_S + 32 * half, tDP = trow + T_DP + 32 * half;
        const uint32_t tP = trow + T_P + 16 * half, tDS = trow + T_DS + 16 * half;
        const uint64_t scale2 = f2_pack(A.scale_log2, A.scale_log2);
        // dQ: this row's query in the tile and head in the group; dK/dV: those of column 32 half + lane
        if (DQ) depend_wait();
        const int own = DQ ? r : 32 * half + lane;
        const int qi = own / A.group, hg = own - qi * A.group;
        float* slot = reinterpret_cast<float*>(gbase + OFF_SLOT) + ew * 64;  // -lse log2(e), D of the 32 columns
        Item it;
        bool ok = true;
#pragma unroll 1
        for (int i = 0; ok && take(i, it); i++) {
            const int64_t head = (int64_t)(it.kh * A.group + hg) * a.total_q;
            float2 ld = make_float2(0.f, 0.f);
            auto load = [&](int n) {  // dK/dV: of the own column of block n
                const int t = it.first + n * A.bq + qi;
                ld = make_float2(0.f, 0.f);
                if (qi < A.bq && t < it.len) ld = A.ld[head + it.s0 + t];
            };
            int n = (it.base & 1) == odd ? 0 : 1;
            if (DQ) {
                if (qi < it.n) ld = A.ld[head + it.r0 + qi];
            } else if (n < it.nb) {
                load(n);
            }
#pragma unroll 1
            for (; n < it.nb; n += 2) {
                const int g = it.base + n;
                const uint32_t ph = (uint32_t)(g >> 1) & 1u;
                if (!DQ) {
                    __syncwarp();  // every lane is done with the previous step's slot
                    slot[lane] = -ld.x;
                    slot[32 + lane] = ld.y;
                    __syncwarp();
                    if (n + 2 < it.nb) load(n + 2);  // in flight meanwhile
                }
                // columns [lo, hi) of this thread's 32 that the row sees, or that see it
                int lo, hi;
                if (DQ) {
                    lo = 0;
                    hi = it.shift + qi - n * BLK - half * 32;
                } else {
                    const int t = it.first + n * A.bq;
                    lo = max(0, it.shift + r - t) * A.group - half * 32;  // (far below 0 the product passes 31 bits)
                    hi = min(A.bq, it.len - t) * A.group - half * 32;
                }
                const bool cut = __any_sync(0xffffffffu, lo > 0 || hi < 32);
                uint32_t v[32];
                if (!(ok = wait(s_full + 8 * odd, ph, abort_flag, status))) break;
                tc_fence_after();
                tc_ld32_issue(tS, v);
                tc_ld_wait(v);
                const ulonglong2* nl4 = reinterpret_cast<const ulonglong2*>(slot);  // four columns a load
                const uint64_t nlr = f2_pack(-ld.x, -ld.x), dr = f2_pack(ld.y, ld.y);
                float p[32];
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    const ulonglong2 nl = DQ ? make_ulonglong2(nlr, nlr) : nl4[c / 4];
                    float x0, x1, x2, x3;
                    f2_unpack(f2_fma(f2_pack(v[c], v[c + 1]), scale2, nl.x), x0, x1);
                    f2_unpack(f2_fma(f2_pack(v[c + 2], v[c + 3]), scale2, nl.y), x2, x3);
                    p[c] = ex2_approx(x0);
                    p[c + 1] = ex2_approx(x1);
                    p[c + 2] = ex2_approx(x2);
                    p[c + 3] = ex2_approx(x3);
                }
                if (cut) {
#pragma unroll
                    for (int c = 0; c < 32; c++)
                        if (c < lo || c >= hi) p[c] = 0.f;
                }
                // P and dS of this parity's previous step have been read
                if (!(ok = wait(ds_free + 8 * odd, ph ^ 1u, abort_flag, status))) break;
                if (!DQ) {
                    tc_fence_after();
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 16; c++) pk[c] = cvt_bf16x2(p[2 * c], p[2 * c + 1]);
                    tc_st16(tP, pk);
                    tc_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full + 8 * odd);
                }
                if (!(ok = wait(dp_full + 8 * odd, ph, abort_flag, status))) break;
                tc_fence_after();
                uint32_t dk[16];
                const ulonglong2* d4 = reinterpret_cast<const ulonglong2*>(slot + 32);
#pragma unroll
                for (int hh = 0; hh < 2; hh++) {
                    uint32_t w[16];
                    tc_ld16_issue(tDP + 16 * hh, w);
                    tc_ld16_wait(w);
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        const int e = 16 * hh + c;
                        const ulonglong2 dd = DQ ? make_ulonglong2(dr, dr) : d4[e / 4];
                        float d0, d1, d2, d3;
                        f2_unpack(f2_mul(f2_pack(p[e], p[e + 1]), f2_sub(f2_pack(w[c], w[c + 1]), dd.x)), d0, d1);
                        f2_unpack(f2_mul(f2_pack(p[e + 2], p[e + 3]), f2_sub(f2_pack(w[c + 2], w[c + 3]), dd.y)), d2, d3);
                        dk[e / 2] = cvt_bf16x2(d0, d1);
                        dk[e / 2 + 1] = cvt_bf16x2(d2, d3);
                    }
                }
                if (cut) {  // not 0 * NaN either
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const uint32_t keep = ((c >= lo && c < hi) ? 0xFFFFu : 0u) |
                                              ((c + 1 >= lo && c + 1 < hi) ? 0xFFFF0000u : 0u);
                        dk[c / 2] &= keep;
                    }
                }
                tc_st16(tDS, dk);
                tc_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_full + 8 * odd);
            }
        }
    }

    if (!DQ) depend_wait();  // dQ is done when dK, dV are
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

size_t round32(size_t n) { return (n + 31) & ~(size_t)31; }

// dQ's tiles (packed rows against blocks of 64 keys), dK's (128 keys against
// blocks of 64 / group queries).
void make_cuts(int group, PackedCut (&cut)[2]) {
    cut[0] = PackedCut{false, 128 / group, BLK};
    cut[1] = PackedCut{true, 128, BLK / group};
}

}  // namespace

int attention_packed_bwd_set_wait_limit(long long cycles) { return set_wait_limit(cycles); }

size_t attention_packed_backward_tc_scratch(int n_seq, int total_q, int total_k, int Hq, int Hkv) {
    PackedCut cut[2];
    make_cuts(Hq / Hkv, cut);
    PackedAttn a = {};
    a.total_q = total_q;
    a.total_k = total_k;
    a.n_seq = n_seq;
    size_t n = round32((size_t)Hq * total_q * sizeof(float2));
    for (int i = 0; i < 2; i++)
        if (cut[i].slots(a) <= PACKED_PLAN_MAX) n += packed_plan_bytes(cut[i].slots(a));
    return n;
}

int launch_attention_packed_backward_tc(const PackedAttn& a, const PackedAttnGrad& g, void* scratch, cudaStream_t s) {
    Args A;
    A.a = a;
    A.g = g;
    A.group = a.Hq / a.Hkv;
    A.scale = 1.f / sqrtf((float)HD);
    A.scale_log2 = LOG2E * A.scale;
    float2* ld = (float2*)scratch;
    A.ld = ld;
    PackedCut cut[2];
    make_cuts(A.group, cut);
    // plans for both, or for neither: they share the launch that sorts them
    PackedPlan* plan[2] = {nullptr, nullptr};
    if (planned(cut[0].slots(a), a.Hkv) && planned(cut[1].slots(a), a.Hkv)) {
        plan[0] = (PackedPlan*)((char*)scratch + round32((size_t)a.Hq * a.total_q * sizeof(float2)));
        plan[1] = (PackedPlan*)((char*)plan[0] + packed_plan_bytes(cut[0].slots(a)));
    }
    // a side without rows is never loaded: any valid address does for its maps
    const bool hq = a.total_q > 0, hk = a.total_k > 0;
    const int nq = hq ? a.total_q : 1, nk = hk ? a.total_k : 1, qt = 128 / A.group, qb = BLK / A.group;
    const void *q = hq ? a.q : a.k, *dy = hq ? g.dout : a.k, *k = hk ? a.k : a.q, *v = hk ? a.v : a.q;
    const int64_t sq = hq ? a.q_stride : a.k_stride, sy = hq ? g.dout_stride : a.k_stride;
    const int64_t sk = hk ? a.k_stride : a.q_stride, sv = hk ? a.v_stride : a.q_stride;
    CUtensorMap q128, y128, q64, y64, k128, v128, k64, v64;
    if (!rows_map(&q128, q, a.Hq, nq, sq, A.group, qt) || !rows_map(&y128, dy, a.Hq, nq, sy, A.group, qt) ||
        !rows_map(&q64, q, a.Hq, nq, sq, A.group, qb) || !rows_map(&y64, dy, a.Hq, nq, sy, A.group, qb) ||
        !rows_map(&k128, k, a.Hkv, nk, sk, 1, 128) || !rows_map(&v128, v, a.Hkv, nk, sv, 1, 128) ||
        !rows_map(&k64, k, a.Hkv, nk, sk, 1, BLK) || !rows_map(&v64, v, a.Hkv, nk, sv, 1, BLK))
        return GPT2_ERR_CUDA;
    if (smem_attr((const void*)packed_bwd_tc_kernel<true>, SMEM) != cudaSuccess ||
        smem_attr((const void*)packed_bwd_tc_kernel<false>, SMEM) != cudaSuccess)
        return GPT2_ERR_CUDA;
    int launches = 0;
    if (plan[0]) {
        const PlanArgs P = {a, {cut[0], cut[1]}, {plan[0], plan[1]}};
        packed_plans_kernel<<<2, 1024, 0, s>>>(P);
        launches++;
    }
    if (hq) {
        const int blocks = (int)(((int64_t)a.total_q * a.Hq + PREP - 1) / PREP);
        // (after anything but the sort, a launch like any other: what it reads has to be complete)
        if (!plan[0]) packed_prep_kernel<<<blocks, 256, 0, s>>>(a, g, ld);
        else if (launch_dependent(packed_prep_kernel, blocks, 256, 0, s, a, g, ld) != cudaSuccess) return GPT2_ERR_CUDA;
        launches++;
    }
    const int sms = gpt2_num_sms();
    for (int i = 0; i < 2; i++) {
        A.cut = cut[i];
        A.plan = plan[i];
        A.items = cut[i].slots(a) * a.Hkv;
        const int grid = A.items < sms ? A.items : sms;
        if (i == 0) {
            A.bq = BLK;
            if (!launches) packed_bwd_tc_kernel<true><<<grid, THREADS, SMEM, s>>>(q128, y128, k64, v64, A);
            else if (launch_dependent(packed_bwd_tc_kernel<true>, grid, THREADS, SMEM, s, q128, y128, k64, v64, A) != cudaSuccess)
                return GPT2_ERR_CUDA;
        } else {
            A.bq = qb;
            if (launch_dependent(packed_bwd_tc_kernel<false>, grid, THREADS, SMEM, s, k128, v128, q64, y64, A) != cudaSuccess)
                return GPT2_ERR_CUDA;
        }
        launches++;
    }
    return launches;
}
