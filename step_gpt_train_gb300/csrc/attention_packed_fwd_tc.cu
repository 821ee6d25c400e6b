// Packed causal attention forward on the tcgen05 tensor cores (bf16, head
// size 64, grouped heads).
//
// The `group` query heads that share a key head are laid into the rows of one
// query tile: row r of a tile is query r / group, head r % group, so one K / V
// block serves the whole group and short prompts still fill the 128 rows (a
// TMA box of 64 x group x 128/group values brings them in this order). A work
// item is a key head and two such tiles, neighbours in one sequence, that
// share every K and V block: at 128 rows a block's loads (32 KB for 2 * 128 *
// 128 * 64 FMA each way) would ask more of the L2 than it gives.
//
// Persistent, one CTA per SM. Per tile and key block:
//   S = Q K^T          tcgen05.mma M=128 N=128 K=64 into TMEM;
//   P = exp2(S log2(e)/sqrt(hd) - m) with a per-row reference m that moves only
//                      when the maximum grows by more than 8 (log2 units), in
//                      fp32; back to TMEM as bf16 pairs (its one rounding);
//   O += P V           tcgen05.mma with P from TMEM as the A operand.
// Two threads share a row, 64 keys each: they exchange their maxima through
// shared memory and keep their own sums. 16 softmax warps (two tiles of eight)
// hide each other's latencies. O moves with m (rarely) in TMEM; at the end of
// an item it is normalised and leaves through a swizzled staging buffer.
//
// Warps: 0 TMA producer; 1, 2 MMA issue for tile 0, 1 (S of the next step
// before PV of the current one); 3 finds the work items (a ring of four in
// shared memory) and zeroes the rows of a V block behind the sequence's end
// (0 * NaN from a neighbour would reach O); 4..19 softmax. Every wait is
// bounded.
#include "attention_packed_tc.cuh"

namespace {

using namespace packed_tc;

constexpr int NST = 3;              // K and V stages
constexpr int NIT = 4;              // work item ring
constexpr int SOFT = 16;            // softmax warps
constexpr int THREADS = 32 * (4 + SOFT);
constexpr float RESCALE = 8.f;      // log2 of the largest P before the reference max moves
// TMEM columns: S of tile 0, 1 | P of tile 0, 1 (bf16 pairs) | O of tile 0, 1
constexpr uint32_t C_S = 0, C_P = 256, C_O = 384;
// shared memory: Q [2 buffers][2 tiles] | K [NST] | V [NST] | staging per softmax warp | exchange | items | barriers
constexpr int OFF_K = 4 * TILE, OFF_V = OFF_K + NST * TILE, OFF_STG = OFF_V + NST * TILE;
constexpr int STG = 32 * 64;        // 32 half rows of O
constexpr int OFF_X = OFF_STG + SOFT * STG;           // [2 steps][2 tiles][2 halves][128] floats
constexpr int OFF_IT = OFF_X + 2 * 2 * 2 * 128 * 4;
constexpr int OFF_BAR = OFF_IT + NIT * 64;
constexpr int SMEM = OFF_BAR + 512 + 1024;
static_assert(SMEM <= 232448, "shared memory per CTA");

struct Item {
    int valid, kh;        // key head
    int q0, nq0, nq1;     // first query row of the buffer; queries of tile 0 and 1
    int k0, lk, vis;      // first key row, keys of the sequence, keys that the first query sees (may be negative)
    int n0, n1, base;     // key blocks of tile 0 and 1; block counter before the item
};
static_assert(sizeof(Item) <= 64, "item slot");

struct Args {
    PackedAttn a;
    int group, qt;        // query heads per key head, queries per tile (128 / group)
    int items;
    float scale_log2;     // log2(e) / sqrt(hd)
};

// No use of these 16 values is scheduled before this point.
__device__ __forceinline__ void hold16(uint32_t* r) {
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]));
}

__global__ void __launch_bounds__(THREADS, 1)
    packed_fwd_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Args A) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const PackedAttn& a = A.a;
    auto sQ = [&](int buf, int t) { return base + (2 * buf + t) * TILE; };
    auto sK = [&](int st) { return base + OFF_K + st * TILE; };
    auto sV = [&](int st) { return base + OFF_V + st * TILE; };
    const uint32_t bars = base + OFF_BAR;
    int nb = 0;
    auto bar = [&](int n) { const uint32_t b = bars + 8u * nb; nb += n; return b; };
    const uint32_t it_full = bar(NIT), it_empty = bar(NIT), q_full = bar(2), q_empty = bar(2);
    const uint32_t k_full = bar(NST), k_empty = bar(NST), v_full = bar(NST), v_empty = bar(NST), v_raw = bar(NST);
    const uint32_t s_full = bar(2), s_free = bar(2), p_full = bar(2), p_free = bar(2), o_done = bar(2), o_free = bar(2);
    const uint32_t xch = bar(8), drain = bar(2);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + OFF_BAR + 496);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + OFF_BAR + 500);
    Item* ring = reinterpret_cast<Item*>(gbase + OFF_IT);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    int* status = a.status;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NIT; i++) {
            mbar_init(it_full + 8 * i, 1);
            mbar_init(it_empty + 8 * i, 3 + SOFT);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(q_full + 8 * i, 1);
            mbar_init(q_empty + 8 * i, 2);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(s_free + 8 * i, SOFT / 2);
            mbar_init(p_full + 8 * i, SOFT / 2);
            mbar_init(p_free + 8 * i, 1);
            mbar_init(o_done + 8 * i, 1);
            mbar_init(o_free + 8 * i, SOFT / 2);
            mbar_init(drain + 8 * i, 1);
        }
        for (int i = 0; i < NST; i++) {
            mbar_init(k_full + 8 * i, 1);
            mbar_init(k_empty + 8 * i, 2);
            mbar_init(v_full + 8 * i, 1);
            mbar_init(v_empty + 8 * i, 2);
            mbar_init(v_raw + 8 * i, 1);
        }
        for (int i = 0; i < 8; i++) mbar_init(xch + 8 * i, 2);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 3) tmem_alloc(smem_addr((const void*)tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // Item i of this CTA's list, by a whole warp; false when the CTA gave up.
    auto take = [&](int i, Item& it) -> bool {
        const int sl = i % NIT;
        if (!warp_wait(it_full + 8 * sl, (i / NIT) & 1, abort_flag, status)) return false;
        it = ring[sl];
        __syncwarp();
        if (lane == 0) mbar_arrive(it_empty + 8 * sl);
        return it.valid;
    };

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        int q_issued[2] = {-1, -1}, k_issued[NST], v_issued[NST], r_uses[NST];
        for (int i = 0; i < NST; i++) k_issued[i] = v_issued[i] = -1, r_uses[i] = 0;
        Item it;
        bool ok = true;
        for (int i = 0; ok && take(i, it); i++) {
            if (lane == 0) {
                const int buf = i & 1;
                const uint32_t qph = (uint32_t)(i >> 1) & 1u;
                ok = mbar_wait(q_empty + 8 * buf, qph ^ 1u, abort_flag, status);
                if (ok) {
                    const uint32_t box = (uint32_t)(A.qt * A.group * HD * 2);
                    mbar_expect_tx(q_full + 8 * buf, it.nq1 > 0 ? 2 * box : box);
                    tma_load_3d(sQ(buf, 0), &tm_q, q_full + 8 * buf, 0, it.kh * A.group, it.q0);
                    if (it.nq1 > 0) tma_load_3d(sQ(buf, 1), &tm_q, q_full + 8 * buf, 0, it.kh * A.group, it.q0 + A.qt);
                    q_issued[buf] = (int)qph;
                    // a tile without blocks does not come for its Q, nor for blocks it does not see
                    if (it.n0 == 0) mbar_arrive(q_empty + 8 * buf);
                    if (it.n1 == 0) mbar_arrive(q_empty + 8 * buf);
                }
                const int n = max(it.n0, it.n1);
                for (int j = 0; ok && j < n; j++) {
                    const int g = it.base + j, st = g % NST;
                    const uint32_t ph = (uint32_t)(g / NST) & 1u;
                    if (!(ok = mbar_wait(k_empty + 8 * st, ph ^ 1u, abort_flag, status))) break;
                    mbar_expect_tx(k_full + 8 * st, TILE);
                    tma_load_3d(sK(st), &tm_k, k_full + 8 * st, 0, it.kh, it.k0 + j * 128);
                    k_issued[st] = (int)ph;
                    if (j >= it.n0) mbar_arrive(k_empty + 8 * st);
                    if (j >= it.n1) mbar_arrive(k_empty + 8 * st);
                    if (!(ok = mbar_wait(v_empty + 8 * st, ph ^ 1u, abort_flag, status))) break;
                    const bool tail = (j + 1) * 128 > it.lk;  // rows of no key: by way of the warp that zeroes them
                    const uint32_t vb = (tail ? v_raw : v_full) + 8 * st;
                    mbar_expect_tx(vb, TILE);
                    tma_load_3d(sV(st), &tm_v, vb, 0, it.kh, it.k0 + j * 128);
                    r_uses[st] += tail;
                    v_issued[st] = tail ? -1 : (int)ph;  // the stage's earlier loads have been read
                    if (j >= it.n0) mbar_arrive(v_empty + 8 * st);
                    if (j >= it.n1) mbar_arrive(v_empty + 8 * st);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        if (lane == 0) {
            for (int b = 0; b < 2; b++)
                if (q_issued[b] >= 0) mbar_drain(q_full + 8 * b, (uint32_t)q_issued[b], status);
            for (int st = 0; st < NST; st++) {
                if (k_issued[st] >= 0) mbar_drain(k_full + 8 * st, (uint32_t)k_issued[st], status);
                if (v_issued[st] >= 0) mbar_drain(v_full + 8 * st, (uint32_t)v_issued[st], status);
                if (r_uses[st]) mbar_drain(v_raw + 8 * st, (uint32_t)(r_uses[st] - 1) & 1u, status);
            }
        }
        __syncwarp();
    } else if (warp <= 2) {
        // ------------------------------------------------------ MMA issue of tile t: the whole warp
        // runs the schedule, one elected lane issues
        const int t = warp - 1;
        const bool leader = elect_one();
        constexpr uint32_t idesc_s = make_idesc(128, 128, false, false);
        constexpr uint32_t idesc_o = make_idesc(128, HD, false, true);
        const uint32_t tS = tmem + C_S + 128 * t, tP = tmem + C_P + 64 * t, tO = tmem + C_O + 64 * t;
        struct Cur {
            bool valid;
            int i, j, n, base;  // item, block, blocks, block counter of block 0
        };
        // The tile's first step at or after item i, looking at no more than `most` items; `on` says whether
        // there are more. An item's ring slot comes free only after its PV, so before a PV is issued only the
        // item after it may be waited for.
        bool on = true;
        auto first_of = [&](int i, int most) -> Cur {
            Item it;
            for (; most > 0 && (on = take(i, it)); i++, most--) {
                const int n = t ? it.n1 : it.n0;
                if (n) return Cur{true, i, 0, n, it.base};
            }
            return Cur{false, i, 0, 0, 0};
        };
        auto issue_s = [&](const Cur& c, int g) -> bool {
            const int b = c.base + c.j, st = b % NST;
            if (c.j == 0 && !warp_wait(q_full + 8 * (c.i & 1), (c.i >> 1) & 1, abort_flag, status)) return false;
            if (!warp_wait(k_full + 8 * st, (b / NST) & 1, abort_flag, status)) return false;
            if (!warp_wait(s_free + 8 * t, (g & 1) ^ 1u, abort_flag, status)) return false;
            tc_fence_after();
            const uint64_t da = sw128_desc(sQ(c.i & 1, t), 16, 1024), db = sw128_desc(sK(st), 16, 1024);
            if (leader) {
#pragma unroll
                for (int k = 0; k < HD / 16; k++) tc_mma(tS, da + 2 * k, db + 2 * k, idesc_s, k > 0 ? 1u : 0u);
                tc_commit(s_full + 8 * t);
                tc_commit(k_empty + 8 * st);
                if (c.j == c.n - 1) tc_commit(q_empty + 8 * (c.i & 1));
            }
            __syncwarp();
            return true;
        };
        constexpr int ALL = 0x7fffffff;
        Cur c = first_of(0, ALL);
        bool ok = !c.valid || issue_s(c, 0);
        int g = 0, done = 0;  // steps, finished items of this tile
        while (ok && c.valid) {
            Cur nx = c;
            if (++nx.j == nx.n) nx = first_of(c.i + 1, 1);
            if (nx.valid && !(ok = issue_s(nx, g + 1))) break;
            const int b = c.base + c.j, st = b % NST;
            if (!(ok = warp_wait(p_full + 8 * t, g & 1, abort_flag, status))) break;
            if (!(ok = warp_wait(v_full + 8 * st, (b / NST) & 1, abort_flag, status))) break;
            if (c.j == 0 && !(ok = warp_wait(o_free + 8 * t, (done & 1) ^ 1u, abort_flag, status))) break;
            tc_fence_after();
            const uint64_t dv = sw128_desc(sV(st), 8192, 1024);
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < 8; kk++)
                    tc_mma_ts(tO, tP + kk * 8, dv + 128 * kk, idesc_o, (c.j > 0 || kk > 0) ? 1u : 0u);
                tc_commit(p_free + 8 * t);
                tc_commit(v_empty + 8 * st);
                if (c.j == c.n - 1) tc_commit(o_done + 8 * t);
            }
            __syncwarp();
            if (c.j == c.n - 1) done++;
            if (!nx.valid && on) {
                nx = first_of(nx.i, ALL);
                if (nx.valid && !(ok = issue_s(nx, g + 1))) break;
            }
            c = nx;
            g++;
        }
        if (leader) tc_commit(drain + 8 * t);
        mbar_drain(drain + 8 * t, 0, status);
    } else if (warp == 3) {
        // ------------------------------------------------------ work items, tails of V
        const int per = 2 * A.qt;
        const int slots = A.items / a.Hkv;
        int x = blockIdx.x, blocks = 0;
        if (blockIdx.x == 0) packed_check(a, lane, 32);
        auto put = [&](int i, Item& it) -> bool {  // the next item with queries, or the end, into ring slot i
            it.valid = 0;
            for (; x < A.items; x += gridDim.x) {
                int f;
                const int slot = slots - 1 - x / a.Hkv;  // the later tiles of a sequence, which see more keys, first
                const int s = find_slot(a.cu_q, a.n_seq, a.total_q, per, slot, f);
                if (s < 0) continue;
                const PackedSeq p = packed_seq(a, s);
                const int at = (slot - f) * per;
                if (at < 0 || at >= p.lq) continue;
                it.valid = 1;
                it.kh = x % a.Hkv;
                it.q0 = p.q0 + at;
                it.nq0 = min(A.qt, p.lq - at);
                it.nq1 = min(A.qt, max(0, p.lq - at - A.qt));
                it.k0 = p.k0;
                it.lk = p.lk;
                it.vis = at + 1 + p.lk - p.lq;
                it.n0 = (max(0, it.vis + it.nq0 - 1) + 127) / 128;
                it.n1 = it.nq1 > 0 ? (max(0, it.vis + A.qt + it.nq1 - 1) + 127) / 128 : 0;
                it.base = blocks;
                blocks += max(it.n0, it.n1);
                x += gridDim.x;
                break;
            }
            const int sl = i % NIT;
            if (!warp_wait(it_empty + 8 * sl, ((i / NIT) & 1) ^ 1u, abort_flag, status)) return false;
            if (lane == 0) {
                ring[sl] = it;
                mbar_arrive(it_full + 8 * sl);
            }
            __syncwarp();
            return true;
        };
        int uses[NST];
        for (int i = 0; i < NST; i++) uses[i] = 0;
        Item cur, nxt;
        bool ok = put(0, cur);
        for (int i = 0; ok && cur.valid; i++) {
            ok = put(i + 1, nxt);
            const int n = max(cur.n0, cur.n1);
            if (ok && n * 128 > cur.lk && n) {
                const int st = (cur.base + n - 1) % NST;
                int u = 0;
#pragma unroll
                for (int e = 0; e < NST; e++)
                    if (e == st) u = uses[e]++;
                if (!(ok = warp_wait(v_raw + 8 * st, u & 1, abort_flag, status))) break;
                zero_rows(gbase + OFF_V + st * TILE, cur.lk - (n - 1) * 128, lane);
                if (lane == 0) mbar_arrive(v_full + 8 * st);
            }
            cur = nxt;
        }
    } else {
        // ------------------------------------------------------ softmax
        const int sw = warp - 4, t = sw >> 3, half = (sw >> 2) & 1, quad = warp & 3;
        const int r = quad * 32 + lane;  // row of the tile = TMEM lane
        const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t tS = trow + C_S + 128 * t + 64 * half, tP = trow + C_P + 64 * t + 32 * half;
        const uint32_t tO = trow + C_O + 64 * t + 32 * half;
        const uint32_t xbar = xch + 8 * (t * 4 + quad);
        float* xs = reinterpret_cast<float*>(gbase + OFF_X) + t * 256;  // [step & 1][..][half][row]
        const int qi = r / A.group, hg = r - qi * A.group;              // this row's query in the tile, head in the group
        const uint64_t scale2 = f2_pack(A.scale_log2, A.scale_log2);
        int g = 0, xc = 0, done = 0;  // steps, exchanges, finished items with blocks
        // this row's value of the other half's thread
        auto exchange = [&](float mine, float& theirs) -> bool {
            float* at = xs + (xc & 1) * 512;
            at[half * 128 + r] = mine;
            __syncwarp();
            if (lane == 0) mbar_arrive(xbar);
            if (!warp_wait(xbar, xc & 1, abort_flag, status)) return false;
            theirs = at[(half ^ 1) * 128 + r];
            xc++;
            return true;
        };
        bool ok = true;
#pragma unroll 1
        for (int i = 0;; i++) {
            // the item stays in the ring until its end, so that its fields take no registers meanwhile
            const int sl = i % NIT;
            if (!warp_wait(it_full + 8 * sl, (i / NIT) & 1, abort_flag, status)) break;
            const volatile Item& it = ring[sl];
            if (!it.valid) break;
            const int n = t ? it.n1 : it.n0;
            const int vis = it.vis + (t ? A.qt : 0) + qi;  // keys that this row sees
            float m = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int j = 0; j < n; j++, g++) {
                uint32_t v[2][32];
                if (!(ok = warp_wait(s_full + 8 * t, g & 1, abort_flag, status))) break;
                tc_fence_after();
                tc_ld32_issue(tS, v[0]);
                tc_ld32_issue(tS + 32, v[1]);
                tc_ld_wait(v[0]);
                tc_ld_wait(v[1]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free + 8 * t);  // the MMA may write the next S
                const int hi = vis - j * 128 - half * 64;    // columns [0, hi) are seen
                if (__any_sync(0xffffffffu, hi < 64)) {
#pragma unroll
                    for (int e = 0; e < 64; e++)
                        if (e >= hi) v[e >> 5][e & 31] = 0xff800000u;
                }
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 64; e += 2)
                    m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], __uint_as_float(v[e >> 5][e & 31]),
                                             __uint_as_float(v[e >> 5][(e & 31) + 1]));
                float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), other;
                if (!(ok = exchange(mx, other))) break;
                mx = fmaxf(mx, other) * A.scale_log2;
                float factor = 1.f;
                const bool move = mx > m + RESCALE;
                if (move) {
                    factor = ex2_approx(m - mx);  // 0 from -inf
                    m = mx;
                    l *= factor;
                }
                const uint64_t nm2 = f2_pack(-m, -m);
                uint64_t l2[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    if (e % 16 == 0) hold16(&v[e >> 5][e & 31]);  // 16 scores at a time: the registers do not suffice for more
                    float x0, x1;
                    f2_unpack(f2_fma(f2_pack(v[e >> 5][e & 31], v[e >> 5][(e & 31) + 1]), scale2, nm2), x0, x1);
                    const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                    l2[(e >> 1) & 1] = f2_add(l2[(e >> 1) & 1], f2_pack(p0, p1));
                    v[0][e / 2] = cvt_bf16x2(p0, p1);
                }
                float s0, s1, s2, s3;
                f2_unpack(l2[0], s0, s1);
                f2_unpack(l2[1], s2, s3);
                l += (s0 + s1) + (s2 + s3);
                // PV of the previous step has finished with P and O
                if (!(ok = warp_wait(p_free + 8 * t, (g & 1) ^ 1u, abort_flag, status))) break;
                tc_fence_after();
                if (j > 0 && __any_sync(0xffffffffu, move)) {
                    uint32_t ov[32];
                    tc_ld32_issue(tO, ov);
                    tc_ld_wait(ov);
#pragma unroll
                    for (int e = 0; e < 32; e++) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * factor);
                    tc_st32(tO, ov);
                }
                tc_st32(tP, v[0]);
                tc_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * t);
            }
            if (!ok) break;
            uint32_t ov[32];
            float other = 0.f;
            if (n) {
                if (!(ok = exchange(l, other))) break;
                if (!(ok = warp_wait(o_done + 8 * t, done & 1, abort_flag, status))) break;
                done++;
                tc_fence_after();
                tc_ld32_issue(tO, ov);
                tc_ld_wait(ov);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_free + 8 * t);
            } else {
#pragma unroll
                for (int e = 0; e < 32; e++) ov[e] = 0;
            }
            const int nq = t ? it.nq1 : it.nq0, row0 = it.q0 + (t ? A.qt : 0), head0 = it.kh * A.group;
            __syncwarp();
            if (lane == 0) mbar_arrive(it_empty + 8 * sl);
            if (nq > 0) {
                // O / l through this warp's staging buffer (half rows of 64 bytes), so that
                // each store covers whole 64-byte pieces of 8 rows
                const bool some = n && vis > 0;
                l += other;
                const float inv = 1.f / l;
                uint8_t* st = gbase + OFF_STG + sw * STG;
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    uint4 w;
                    uint32_t* wp = &w.x;
#pragma unroll
                    for (int u = 0; u < 4; u++)
                        wp[u] = some ? cvt_bf16x2(__uint_as_float(ov[q * 8 + 2 * u]) * inv,
                                                  __uint_as_float(ov[q * 8 + 2 * u + 1]) * inv)
                                     : 0u;
                    stage16(st, lane, q, w);
                }
                __syncwarp();
                bf16* o = reinterpret_cast<bf16*>(a.o);
#pragma unroll 1
                for (int e = 0; e < 4; e++) {
                    const int sr = e * 8 + (lane >> 2), c = lane & 3;
                    const int rr = quad * 32 + sr, q = rr / A.group, h = rr - q * A.group;
                    if (q < nq)
                        *reinterpret_cast<uint4*>(o + (int64_t)(row0 + q) * a.o_stride + (head0 + h) * HD +
                                                  half * 32 + c * 8) =
                            *reinterpret_cast<const uint4*>(st + sr * 64 + ((c ^ ((sr >> 1) & 3)) << 4));
                }
                if (half == 0 && qi < nq)
                    a.lse[(int64_t)(head0 + hg) * a.total_q + row0 + qi] =
                        some ? (m + log2f(l)) * LN2 : -INFINITY;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 3) {
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

int attention_packed_fwd_set_wait_limit(long long cycles) { return set_wait_limit(cycles); }

int launch_attention_packed_forward_tc(const PackedAttn& a, cudaStream_t s) {
    Args A;
    A.a = a;
    A.group = a.Hq / a.Hkv;
    A.qt = 128 / A.group;
    A.items = (a.total_q / (2 * A.qt) + a.n_seq) * a.Hkv;
    A.scale_log2 = LOG2E / sqrtf((float)HD);
    CUtensorMap mq, mk, mv;
    // without keys nothing is loaded through the key and value maps
    const bool keys = a.total_k > 0;
    if (!rows_map(&mq, a.q, a.Hq, a.total_q, a.q_stride, A.group, A.qt) ||
        !rows_map(&mk, keys ? a.k : a.q, a.Hkv, keys ? a.total_k : 1, keys ? a.k_stride : a.q_stride, 1, 128) ||
        !rows_map(&mv, keys ? a.v : a.q, a.Hkv, keys ? a.total_k : 1, keys ? a.v_stride : a.q_stride, 1, 128))
        return GPT2_ERR_CUDA;
    if (smem_attr((const void*)packed_fwd_tc_kernel, SMEM) != cudaSuccess) return GPT2_ERR_CUDA;
    const int grid = A.items < gpt2_num_sms() ? A.items : gpt2_num_sms();
    packed_fwd_tc_kernel<<<grid, THREADS, SMEM, s>>>(mq, mk, mv, A);
    return 1;
}
