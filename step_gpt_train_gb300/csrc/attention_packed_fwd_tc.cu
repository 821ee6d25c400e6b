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
//   P = exp2(S log2(e)/sqrt(hd) - m) in fp32, m the row's maximum in its first
//                      block; back to TMEM as bf16 pairs (its one rounding);
//   O += P V           tcgen05.mma with P from TMEM as the A operand.
// One thread per row, 128 scores in its registers: two threads per row with 64
// each (16 softmax warps) exchanged their maxima and spent 470 instructions a
// warp and step where this form spends about as many for twice the scores.
//
// P, the sum l and O are floating-point numbers, precise at any scale, so m
// needs to be the maximum only to within fp32's range: later blocks are not
// searched for a larger one (which took a seventh of a step), and O never
// moves. Where a row's l is not between 1 and 2^40 at the end (scores that grow
// by 28 over the first block's, infinities, NaN), or its first block's scores
// are all -inf, the output warps mark its item. A CTA that has marked ones goes
// through the whole schedule once more with those, m then being a running
// maximum: where it grows by more than 8 (log2 units) the softmax threads scale
// O in TMEM before the next PV. Scores that grow in every row cost 2.5 to 3.4
// times the call (16 heads on 4: 4096 tokens 78 and 195 us, 16384 0.48 and 1.6
// ms). The second pass is code of its own, each role's behind its first: one
// loop for both took 75 us for the documents below instead of 71, a launch of
// its own 4 us more for the smallest calls.
//
// Warps: 0 TMA producer; 1, 2 MMA issue for tile 0, 1 (S of the next step
// before PV of the current one); 3 finds the work items (a ring of two in
// shared memory) and zeroes the rows of a V block behind the sequence's end
// (0 * NaN from a neighbour would reach O); 4..7 output, so that the softmax
// warps go on with the next item (short documents spent more on the way out
// than on their blocks); 8..15 softmax. Registers: 184 a thread for the
// softmax warps, 72 for the others. Every wait is bounded.
//
// Measured: 62 documents of 100 to 1024 tokens, 12 heads, 71 us; 16 prompts of
// up to 4096 tokens, 16 heads on 4, 95 us (75 GFLOP: 785 TFLOP/s). Long
// sequences are bound by the softmax warps' chain of about 2000 cycles a block
// (wait, 128 scores from TMEM, exponentials, P back), two such warps to a
// scheduler: 63 pairs of blocks a CTA on the prompts. The documents are ten items
// a CTA and 32 pairs of blocks, half of their time; the rest is what an item
// costs from its draw to its first scores and from its last P to O. The
// exponential unit alone would take 17 and 44 us, the tensor cores 10 and 38.
#include "attention_packed_tc.cuh"

#include <type_traits>

namespace {

using namespace packed_tc;

constexpr int NST = 4;              // K and V stages
constexpr int NIT = 2;              // work item ring: an item is drawn when the one before it begins, not earlier
constexpr int SOFT = 8;             // softmax warps, four to a tile
constexpr int THREADS = 32 * (8 + SOFT);
constexpr int REGS_SOFT = 184, REGS_REST = 72;  // 256 * 184 + 256 * 72 = the 65536 of the launch (128 a thread)
constexpr float MOST = 0x1p40f;     // sum of a row's weights up to which its first block's maximum serves
constexpr float RESCALE = 8.f;      // log2 units that a running maximum may lag behind
// TMEM columns: S of tile 0, 1 | P of tile 0, 1 (bf16 pairs) | O of tile 0, 1
constexpr uint32_t C_S = 0, C_P = 256, C_O = 384;
// shared memory: Q [2 buffers][2 tiles] | K [NST] | V [NST] | staging per output warp | m, l | items | barriers
constexpr int OFF_K = 4 * TILE, OFF_V = OFF_K + NST * TILE, OFF_STG = OFF_V + NST * TILE;
constexpr int STG = 32 * 128;       // 32 rows of O
constexpr int OFF_ML = OFF_STG + 4 * STG;  // [2 tiles][m, l][128] floats
constexpr int OFF_IT = OFF_ML + 2 * 2 * 128 * 4;
constexpr int OFF_MARK = OFF_IT + NIT * 64;
constexpr int BARS = 46, OFF_BAR = OFF_MARK + 64;  // a set for each pass
constexpr int OFF_SLOT = OFF_BAR + 2 * BARS * 8;   // TMEM address, abort flag
constexpr int SMEM = OFF_SLOT + 16 + 1024;
static_assert(SMEM <= 232448, "shared memory per CTA");

struct Item {
    int valid, kh;        // key head
    int q0, nq0, nq1;     // first query row of the buffer; queries of tile 0 and 1
    int k0, lk, vis;      // first key row, keys of the sequence, keys that the first query sees (may be negative)
    int n0, n1, base;     // key blocks of tile 0 and 1; block counter before the item
    int id;               // see next_tile
};
static_assert(sizeof(Item) <= 64, "item slot");

struct Args {
    PackedAttn a;
    int group, qt;        // query heads per key head, queries per tile (128 / group)
    int items;
    float scale_log2;     // log2(e) / sqrt(hd)
    PackedCut cut;        // pairs of tiles, key blocks of 128
    PackedPlan* plan;     // sorted items, or null: found from the offsets
    int* link;            // of a marked item's number: the one marked before it, or -1
};

// A set of barriers.
struct Bars {
    uint32_t at;
    __device__ __forceinline__ uint32_t take(int n) { const uint32_t b = at; at += 8u * n; return b; }
    const uint32_t it_full, it_empty, q_full, q_empty, k_full, k_empty, v_full, v_empty, v_raw;
    const uint32_t s_full, s_free, p_full, p_free, o_done, o_free, l_full, l_empty, drain;
    __device__ __forceinline__ explicit Bars(uint32_t first)
        : at(first), it_full(take(NIT)), it_empty(take(NIT)), q_full(take(2)), q_empty(take(2)), k_full(take(NST)),
          k_empty(take(NST)), v_full(take(NST)), v_empty(take(NST)), v_raw(take(NST)), s_full(take(2)), s_free(take(2)),
          p_full(take(2)), p_free(take(2)), o_done(take(2)), o_free(take(2)), l_full(take(2)), l_empty(take(2)),
          drain(take(2)) {}
    __device__ __forceinline__ void init() const {  // by one thread
        for (int i = 0; i < NIT; i++) {
            mbar_init(it_full + 8 * i, 1);
            mbar_init(it_empty + 8 * i, 3 + 4 + SOFT);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(q_full + 8 * i, 1);
            mbar_init(q_empty + 8 * i, 2);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(s_free + 8 * i, SOFT / 2);
            mbar_init(p_full + 8 * i, SOFT / 2);
            mbar_init(p_free + 8 * i, 1);
            mbar_init(o_done + 8 * i, 1);
            mbar_init(o_free + 8 * i, 4);
            mbar_init(l_full + 8 * i, SOFT / 2);
            mbar_init(l_empty + 8 * i, 4);
            mbar_init(drain + 8 * i, 1);
        }
        for (int i = 0; i < NST; i++) {
            mbar_init(k_full + 8 * i, 1);
            mbar_init(k_empty + 8 * i, 2);
            mbar_init(v_full + 8 * i, 1);
            mbar_init(v_empty + 8 * i, 2);
            mbar_init(v_raw + 8 * i, 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
};
static_assert(2 * NIT + 2 * 11 + 5 * NST == BARS, "barriers of a set");

// The marked items, a list through Args::link by their numbers; and of the
// newest items (i at i % 4: the output warps are at most three apart) which
// is in it, as i + 1.
struct Marks {
    int head, item[4];
};
static_assert(sizeof(Marks) <= 64, "its place");

__global__ void __launch_bounds__(1024) packed_plan_kernel(PackedAttn a, PackedCut cut, PackedPlan* plan) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the forward's blocks may set themselves up
    packed_plan_block(a, cut, plan, true);
}

struct Maps {
    const CUtensorMap *q, *k, *v;
};
enum Role { LOAD, MMA, ITEMS, OUT, SOFTMAX };

// What the warps of a role do in a pass over the CTA's items. The first pass draws them; AGAIN: those that it marked.
template <bool AGAIN, Role ROLE>
__device__ __forceinline__ void run(const Maps& maps, const Args& A, uint32_t base, uint8_t* gbase, uint32_t tmem) {
    const PackedAttn& a = A.a;
    auto sQ = [&](int buf, int t) { return base + (2 * buf + t) * TILE; };
    auto sK = [&](int st) { return base + OFF_K + st * TILE; };
    auto sV = [&](int st) { return base + OFF_V + st * TILE; };
    const Bars B(base + OFF_BAR + (AGAIN ? BARS * 8 : 0));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + OFF_SLOT + 4);
    Marks& marks = *reinterpret_cast<Marks*>(gbase + OFF_MARK);
    Item* ring = reinterpret_cast<Item*>(gbase + OFF_IT);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    int* status = a.status;

    // Item i of this CTA's list, by a whole warp; false behind the last, or when the CTA gave up.
    auto take = [&](int i, Item& it) -> bool {
        const int sl = i % NIT;
        if (!wait(B.it_full + 8 * sl, (i / NIT) & 1, abort_flag, status)) return false;
        it = ring[sl];
        __syncwarp();
        if (lane == 0) mbar_arrive(B.it_empty + 8 * sl);
        return it.valid;
    };

    if constexpr (ROLE == LOAD) {
        // ------------------------------------------------------ TMA producer
        int q_issued[2] = {-1, -1}, k_issued[NST], v_issued[NST], r_uses[NST];
        for (int i = 0; i < NST; i++) k_issued[i] = v_issued[i] = -1, r_uses[i] = 0;
        Item it;
        bool ok = true;
        for (int i = 0; ok && take(i, it); i++) {
            if (lane == 0) {
                const int buf = i & 1;
                const uint32_t qph = (uint32_t)(i >> 1) & 1u;
                ok = mbar_wait(B.q_empty + 8 * buf, qph ^ 1u, abort_flag, status);
                if (ok) q_issued[buf] = (int)qph;
                if (ok && it.n0 == 0 && it.n1 == 0) {
                    // nobody comes for its Q: none is loaded, whose bytes could still be on their way when the buffer
                    // is filled for the item after the next
                    mbar_arrive(B.q_full + 8 * buf);
                    mbar_arrive(B.q_empty + 8 * buf);
                    mbar_arrive(B.q_empty + 8 * buf);
                } else if (ok) {
                    const uint32_t box = (uint32_t)(A.qt * A.group * HD * 2);
                    mbar_expect_tx(B.q_full + 8 * buf, it.nq1 > 0 ? 2 * box : box);
                    tma_load_3d(sQ(buf, 0), maps.q, B.q_full + 8 * buf, 0, it.kh * A.group, it.q0);
                    if (it.nq1 > 0) tma_load_3d(sQ(buf, 1), maps.q, B.q_full + 8 * buf, 0, it.kh * A.group, it.q0 + A.qt);
                    // a tile without blocks does not come for its Q, nor for blocks it does not see
                    if (it.n0 == 0) mbar_arrive(B.q_empty + 8 * buf);
                    if (it.n1 == 0) mbar_arrive(B.q_empty + 8 * buf);
                }
                const int n = max(it.n0, it.n1);
                for (int j = 0; ok && j < n; j++) {
                    const int g = it.base + j, st = g % NST;
                    const uint32_t ph = (uint32_t)(g / NST) & 1u;
                    if (!(ok = mbar_wait(B.k_empty + 8 * st, ph ^ 1u, abort_flag, status))) break;
                    mbar_expect_tx(B.k_full + 8 * st, TILE);
                    tma_load_3d(sK(st), maps.k, B.k_full + 8 * st, 0, it.kh, it.k0 + j * 128);
                    k_issued[st] = (int)ph;
                    if (j >= it.n0) mbar_arrive(B.k_empty + 8 * st);
                    if (j >= it.n1) mbar_arrive(B.k_empty + 8 * st);
                    if (!(ok = mbar_wait(B.v_empty + 8 * st, ph ^ 1u, abort_flag, status))) break;
                    const bool tail = (j + 1) * 128 > it.lk;  // rows of no key: by way of the warp that zeroes them
                    const uint32_t vb = (tail ? B.v_raw : B.v_full) + 8 * st;
                    mbar_expect_tx(vb, TILE);
                    tma_load_3d(sV(st), maps.v, vb, 0, it.kh, it.k0 + j * 128);
                    r_uses[st] += tail;
                    v_issued[st] = tail ? -1 : (int)ph;  // the stage's earlier loads have been read
                    if (j >= it.n0) mbar_arrive(B.v_empty + 8 * st);
                    if (j >= it.n1) mbar_arrive(B.v_empty + 8 * st);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        if (lane == 0) {
            for (int b = 0; b < 2; b++)
                if (q_issued[b] >= 0) mbar_drain(B.q_full + 8 * b, (uint32_t)q_issued[b], status);
            for (int st = 0; st < NST; st++) {
                if (k_issued[st] >= 0) mbar_drain(B.k_full + 8 * st, (uint32_t)k_issued[st], status);
                if (v_issued[st] >= 0) mbar_drain(B.v_full + 8 * st, (uint32_t)v_issued[st], status);
                if (r_uses[st]) mbar_drain(B.v_raw + 8 * st, (uint32_t)(r_uses[st] - 1) & 1u, status);
            }
        }
        __syncwarp();
    } else if constexpr (ROLE == MMA) {
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
        int k_seen = -1;  // the last key block waited for ahead of its step
        auto issue_s = [&](const Cur& c, int g) -> bool {
            const int b = c.base + c.j, st = b % NST;
            if (c.j == 0 && !wait(B.q_full + 8 * (c.i & 1), (c.i >> 1) & 1, abort_flag, status)) return false;
            if (k_seen != b && !wait(B.k_full + 8 * st, (b / NST) & 1, abort_flag, status)) return false;
            if (!wait(B.s_free + 8 * t, (g & 1) ^ 1u, abort_flag, status)) return false;
            tc_fence_after();
            const uint64_t da = sw128_desc(sQ(c.i & 1, t), 16, 1024), db = sw128_desc(sK(st), 16, 1024);
            if (leader) {
#pragma unroll
                for (int k = 0; k < HD / 16; k++) tc_mma(tS, da + 2 * k, db + 2 * k, idesc_s, k > 0 ? 1u : 0u);
                tc_commit(B.s_full + 8 * t);
                tc_commit(B.k_empty + 8 * st);
                if (c.j == c.n - 1) tc_commit(B.q_empty + 8 * (c.i & 1));
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
            // P last: the others have long arrived, and each wait passed after P would delay PV
            const int b = c.base + c.j, st = b % NST;
            const uint64_t dv = sw128_desc(sV(st), 8192, 1024);
            if (!(ok = wait(B.v_full + 8 * st, (b / NST) & 1, abort_flag, status))) break;
            if (c.j == 0 && !(ok = wait(B.o_free + 8 * t, (done & 1) ^ 1u, abort_flag, status))) break;
            if (nx.valid && nx.j < nx.n - 1) {  // the K block after the next one, for the S that follows this PV
                const int b2 = nx.base + nx.j + 1, st2 = b2 % NST;
                if (!(ok = wait(B.k_full + 8 * st2, (b2 / NST) & 1, abort_flag, status))) break;
                k_seen = b2;
            }
            if (!(ok = wait(B.p_full + 8 * t, g & 1, abort_flag, status))) break;
            tc_fence_after();
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < 8; kk++)
                    tc_mma_ts(tO, tP + kk * 8, dv + 128 * kk, idesc_o, (c.j > 0 || kk > 0) ? 1u : 0u);
                tc_commit(B.p_free + 8 * t);
                tc_commit(B.v_empty + 8 * st);
                if (c.j == c.n - 1) tc_commit(B.o_done + 8 * t);
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
        if (leader) tc_commit(B.drain + 8 * t);
        mbar_drain(B.drain + 8 * t, 0, status);
    } else if constexpr (ROLE == ITEMS) {
        // ------------------------------------------------------ work items, tails of V
        int x = blockIdx.x, blocks = 0;
        if (!AGAIN && blockIdx.x == 0 && !A.plan) packed_check(a, lane, 32);
        if (A.plan) asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is written
        int id = -1;  // of the newest item
        auto put = [&](int i, Item& it) -> bool {  // the next item, or the end, into ring slot i
            PackedTile p;
            if constexpr (AGAIN) {
                id = i == 0 ? marks.head : A.link[id];
                it.valid = id >= 0;
                if (it.valid) tile_of(a, A.cut, A.plan, A.items, id, p, it.kh);
            } else {
                it.valid = next_tile(a, A.cut, A.plan, A.items, x, p, it.kh, &id);
            }
            it.id = id;
            if (it.valid) {
                it.q0 = p.r0;
                it.nq0 = min(A.qt, p.n);
                it.nq1 = p.n - it.nq0;
                it.k0 = p.s0;
                it.lk = p.len;
                it.vis = p.shift;
                it.n0 = A.cut.blocks(p, it.nq0);
                it.n1 = it.nq1 > 0 ? A.cut.blocks(p, p.n) : 0;
                it.base = blocks;
                blocks += max(it.n0, it.n1);
            }
            const int sl = i % NIT;
            if (!wait(B.it_empty + 8 * sl, ((i / NIT) & 1) ^ 1u, abort_flag, status)) return false;
            if (lane == 0) {
                ring[sl] = it;
                mbar_arrive(B.it_full + 8 * sl);
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
                if (!(ok = wait(B.v_raw + 8 * st, u & 1, abort_flag, status))) break;
                zero_rows(gbase + OFF_V + st * TILE, cur.lk - (n - 1) * 128, lane);
                if (lane == 0) mbar_arrive(B.v_full + 8 * st);
            }
            cur = nxt;
        }
    } else if constexpr (ROLE == OUT) {
        // ------------------------------------------------------ output
        const int quad = warp & 3, r = quad * 32 + lane;  // row of a tile = TMEM lane
        const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16) + C_O;
        const float* ml = reinterpret_cast<const float*>(gbase + OFF_ML);
        uint8_t* st = gbase + OFF_STG + quad * STG;
        bf16* o = reinterpret_cast<bf16*>(a.o);
        const int qi = r / A.group, hg = r - qi * A.group;  // this row's query in the tile, head in the group
        int done[2] = {0, 0};
        Item it;
        bool ok = true;
#pragma unroll 1
        for (int i = 0; ok && take(i, it); i++) {
#pragma unroll 1
            for (int t = 0; t < 2; t++) {
                const int n = t ? it.n1 : it.n0, nq = t ? it.nq1 : it.nq0;
                if (nq <= 0) continue;
                const int row = it.q0 + (t ? A.qt : 0) + qi;
                const bool mine = qi < nq;  // (and qi < qt: a tile's unused last rows lie behind its nq queries)
                // out through this warp's staging buffer (chunk c of row s at (c ^ (s & 7)) * 16: conflict-free
                // both ways), so that each store covers four whole 128-byte rows
                const int64_t off = mine ? (int64_t)row * a.o_stride + (it.kh * A.group + hg) * HD : -1;
                uint8_t* my = st + lane * 128;
                float L = -INFINITY;
                if (n) {
                    const int d = t ? done[1]++ : done[0]++;
                    if (!(ok = wait(B.l_full + 8 * t, d & 1, abort_flag, status))) break;
                    const float m = ml[t * 256 + r], l = ml[t * 256 + 128 + r];
                    const int vis = it.vis + (t ? A.qt : 0) + qi;  // keys that the row sees
                    // (m = -inf: no finite score in the first block, so l is against 0 and says nothing)
                    // (m = -inf: no finite score in the first block, so l is against 0 and says nothing)
                    if (!AGAIN && __any_sync(0xffffffffu, mine && vis > 0 && !(m > -INFINITY && l > 0.5f && l < MOST)) &&
                        lane == 0 && atomicExch(&marks.item[i & 3], i + 1) != i + 1)
                        A.link[it.id] = atomicExch(&marks.head, it.id);
                    if (!(ok = wait(B.o_done + 8 * t, d & 1, abort_flag, status))) break;
                    tc_fence_after();
                    const bool some = vis > 0;
                    const float inv = 1.f / l;
#pragma unroll
                    for (int hh = 0; hh < 2; hh++) {
                        uint32_t ov[32];
                        tc_ld32_issue(trow + 64 * t + 32 * hh, ov);
                        tc_ld_wait(ov);
                        if (hh) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) {
                                mbar_arrive(B.o_free + 8 * t);
                                mbar_arrive(B.l_empty + 8 * t);
                            }
                        }
#pragma unroll
                        for (int c = 0; c < 4; c++) {
                            uint32_t w[4];
#pragma unroll
                            for (int u = 0; u < 4; u++)
                                w[u] = some ? cvt_bf16x2(__uint_as_float(ov[c * 8 + 2 * u]) * inv,
                                                         __uint_as_float(ov[c * 8 + 2 * u + 1]) * inv)
                                            : 0u;
                            *reinterpret_cast<uint4*>(my + (((hh * 4 + c) ^ (lane & 7)) << 4)) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    if (some) L = (m + log2f(l)) * LN2;
                } else {
#pragma unroll
                    for (int c = 0; c < 8; c++)
                        *reinterpret_cast<uint4*>(my + (c << 4)) = make_uint4(0, 0, 0, 0);
                }
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int sr = e * 4 + (lane >> 3), c = lane & 7;
                    const int64_t at = __shfl_sync(0xffffffffu, off, sr);
                    const uint4 w = *reinterpret_cast<const uint4*>(st + sr * 128 + ((c ^ (sr & 7)) << 4));
                    if (at >= 0) *reinterpret_cast<uint4*>(o + at + c * 8) = w;
                }
                __syncwarp();  // the staged rows have been read
                if (mine) a.lse[(int64_t)(it.kh * A.group + hg) * a.total_q + row] = L;
            }
        }
    } else if constexpr (ROLE == SOFTMAX) {
        // ------------------------------------------------------ softmax
        const int t = (warp >> 2) & 1, quad = warp & 3;
        const int r = quad * 32 + lane;  // row of the tile = TMEM lane
        const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t tS = trow + C_S + 128 * t, tP = trow + C_P + 64 * t, tO = trow + C_O + 64 * t;
        const int qi = r / A.group;      // this row's query in the tile
        float* ml = reinterpret_cast<float*>(gbase + OFF_ML) + t * 256;
        const uint64_t scale2 = f2_pack(A.scale_log2, A.scale_log2);
        int g = 0, done = 0;             // steps, finished items with blocks
        bool ok = true;
#pragma unroll 1
        for (int i = 0;; i++) {
            // the item stays in the ring until its end, so that its fields take no registers meanwhile
            const int sl = i % NIT;
            if (!wait(B.it_full + 8 * sl, (i / NIT) & 1, abort_flag, status)) break;
            const volatile Item& it = ring[sl];
            if (!it.valid) break;
            const int n = t ? it.n1 : it.n0;
            const int vis = it.vis + (t ? A.qt : 0) + qi;  // keys that this row sees
            float m = -INFINITY, l = 0.f;
            if constexpr (!AGAIN) {
#pragma unroll 1
                for (int j = 0; j < n; j++, g++) {
                    uint32_t v[4][32];
                    if (!(ok = wait(B.s_full + 8 * t, g & 1, abort_flag, status))) break;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < 4; c++) tc_ld32_issue(tS + 32 * c, v[c]);
#pragma unroll
                    for (int c = 0; c < 4; c++) tc_ld_wait(v[c]);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(B.s_free + 8 * t);  // the MMA may write the next S
                    const int hi = vis - j * 128;  // columns [0, hi) are seen
                    if (__any_sync(0xffffffffu, hi < 128)) {
                        // chunks that some row of the warp does not see whole
                        const int least = __reduce_min_sync(0xffffffffu, hi);
#pragma unroll
                        for (int c = 0; c < 4; c++)
                            if (least < c * 32 + 32) {
#pragma unroll
                                for (int e = 0; e < 32; e++)
                                    if (c * 32 + e >= hi) v[c][e] = 0xff800000u;
                            }
                    }
                    if (j == 0) {
                        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int c = 0; c < 4; c++)
#pragma unroll
                            for (int e = 0; e < 32; e += 2)
                                m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], __uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
                        m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * A.scale_log2;
                    }
                    const float nm = m == -INFINITY ? 0.f : -m;
                    const uint64_t nm2 = f2_pack(nm, nm);
                    uint64_t l2[4] = {0, 0, 0, 0};
                    uint32_t pk[2][32];
#pragma unroll
                    for (int c = 0; c < 4; c++)
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float x0, x1;
                            f2_unpack(f2_fma(f2_pack(v[c][e], v[c][e + 1]), scale2, nm2), x0, x1);
                            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                            l2[(e >> 1) & 3] = f2_add(l2[(e >> 1) & 3], f2_pack(p0, p1));
                            pk[c >> 1][(c & 1) * 16 + e / 2] = cvt_bf16x2(p0, p1);
                        }
                    // PV of the previous step has finished with P
                    if (!(ok = wait(B.p_free + 8 * t, (g & 1) ^ 1u, abort_flag, status))) break;
                    tc_fence_after();
                    tc_st32(tP, pk[0]);
                    tc_st32(tP + 32, pk[1]);
                    l += f2_total(f2_add(f2_add(l2[0], l2[1]), f2_add(l2[2], l2[3])));
                    tc_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(B.p_full + 8 * t);
                }
            } else {  // a running maximum; 32 scores at a time
#pragma unroll 1
                for (int j = 0; j < n; j++, g++) {
                    if (!(ok = wait(B.s_full + 8 * t, g & 1, abort_flag, status))) break;
                    tc_fence_after();
                    const int hi = vis - j * 128;
                    uint32_t v[32];
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < 4; c++) {
                        tc_ld32_issue(tS + 32 * c, v);
                        tc_ld_wait(v);
#pragma unroll
                        for (int e = 0; e < 32; e++)
                            if (c * 32 + e < hi) mx = fmaxf(mx, __uint_as_float(v[e]));
                    }
                    mx *= A.scale_log2;
                    const bool move = mx > m + RESCALE;
                    const float factor = move ? ex2_approx(m - mx) : 1.f;  // 0 from -inf
                    m = move ? mx : m;
                    l *= factor;
                    // PV of the previous step has finished with P and O
                    if (!(ok = wait(B.p_free + 8 * t, (g & 1) ^ 1u, abort_flag, status))) break;
                    tc_fence_after();
                    if (j > 0 && __any_sync(0xffffffffu, move)) {
#pragma unroll 1
                        for (int c = 0; c < 2; c++) {
                            tc_ld32_issue(tO + 32 * c, v);
                            tc_ld_wait(v);
#pragma unroll
                            for (int e = 0; e < 32; e++) v[e] = __float_as_uint(__uint_as_float(v[e]) * factor);
                            tc_st32(tO + 32 * c, v);
                        }
                    }
                    const float nm = m == -INFINITY ? 0.f : -m;
#pragma unroll 1
                    for (int c = 0; c < 4; c++) {
                        tc_ld32_issue(tS + 32 * c, v);
                        tc_ld_wait(v);
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float p0 = c * 32 + e < hi ? ex2_approx(fmaf(__uint_as_float(v[e]), A.scale_log2, nm)) : 0.f;
                            const float p1 =
                                c * 32 + e + 1 < hi ? ex2_approx(fmaf(__uint_as_float(v[e + 1]), A.scale_log2, nm)) : 0.f;
                            l += p0 + p1;
                            pk[e / 2] = cvt_bf16x2(p0, p1);
                        }
                        tc_st16(tP + 16 * c, pk);
                    }
                    tc_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(B.s_free + 8 * t);
                        mbar_arrive(B.p_full + 8 * t);
                    }
                }
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(B.it_empty + 8 * sl);
            if (n) {  // m and l to the output warps
                if (!wait(B.l_empty + 8 * t, (done & 1) ^ 1u, abort_flag, status)) break;
                done++;
                ml[r] = m;
                ml[128 + r] = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(B.l_full + 8 * t);
            }
        }
    }
}

__global__ void __launch_bounds__(THREADS, 1)
    packed_fwd_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Args A) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + OFF_SLOT);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + OFF_SLOT + 4);
    volatile Marks& marks = *reinterpret_cast<volatile Marks*>(gbase + OFF_MARK);
    const int warp = threadIdx.x / 32;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int k = 0; k < 4; k++) marks.item[k] = 0;
        marks.head = -1;
        Bars(base + OFF_BAR).init();
    }
    if (warp == 3) tmem_alloc(smem_addr((const void*)tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Maps maps = {&tm_q, &tm_k, &tm_v};

    auto all_sync = [] {
        tc_fence_before();
        asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
        tc_fence_after();
    };
    auto passes = [&](auto first, auto again) {
        first(base, gbase, tmem);
        all_sync();
        if (marks.head < 0 || *abort_flag) return;
        if (threadIdx.x == 0) Bars(base + OFF_BAR + BARS * 8).init();
        all_sync();
        // values that the compiler takes for new ones: what both passes compute from them would stay in registers
        // through the first
        uint32_t b = base, t = tmem;
        uint8_t* g = gbase;
        asm volatile("" : "+r"(b), "+r"(t), "+l"(g));
        again(b, g, t);
        all_sync();
    };
#define PASSES(ROLE)                                                                              \
    passes([&](uint32_t b, uint8_t* g, uint32_t t) { run<false, ROLE>(maps, A, b, g, t); },       \
           [&](uint32_t b, uint8_t* g, uint32_t t) { run<true, ROLE>(maps, A, b, g, t); })
    if (warp < 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));
        if (warp == 0) PASSES(LOAD);
        else if (warp <= 2) PASSES(MMA);
        else if (warp == 3) PASSES(ITEMS);
        else PASSES(OUT);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFT));
        PASSES(SOFTMAX);
    }
#undef PASSES
    if (warp == 3) {
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

int attention_packed_fwd_set_wait_limit(long long cycles) { return set_wait_limit(cycles); }

// The sorted items (where the sort takes them), a link for each item.
static size_t plan_bytes(int slots) { return slots <= PACKED_PLAN_MAX ? packed_plan_bytes(slots) : 0; }
size_t attention_packed_forward_tc_scratch(int n_seq, int total_q, int Hq, int Hkv) {
    const int slots = packed_slots(total_q, n_seq, 2 * (128 / (Hq / Hkv)));
    return plan_bytes(slots) + (size_t)slots * Hkv * 4;
}

int launch_attention_packed_forward_tc(const PackedAttn& a, PackedPlan* plan, cudaStream_t s) {
    Args A;
    A.a = a;
    A.group = a.Hq / a.Hkv;
    A.qt = 128 / A.group;
    A.cut = PackedCut{false, 2 * A.qt, 128};
    A.items = A.cut.slots(a) * a.Hkv;
    A.scale_log2 = LOG2E / sqrtf((float)HD);
    A.plan = planned(A.cut.slots(a), a.Hkv) ? plan : nullptr;
    CUtensorMap mq, mk, mv;
    // without keys nothing is loaded through the key and value maps
    const bool keys = a.total_k > 0;
    if (!rows_map(&mq, a.q, a.Hq, a.total_q, a.q_stride, A.group, A.qt) ||
        !rows_map(&mk, keys ? a.k : a.q, a.Hkv, keys ? a.total_k : 1, keys ? a.k_stride : a.q_stride, 1, 128) ||
        !rows_map(&mv, keys ? a.v : a.q, a.Hkv, keys ? a.total_k : 1, keys ? a.v_stride : a.q_stride, 1, 128))
        return GPT2_ERR_CUDA;
    if (smem_attr((const void*)packed_fwd_tc_kernel, SMEM) != cudaSuccess) return GPT2_ERR_CUDA;
    A.link = (int*)((char*)plan + plan_bytes(A.cut.slots(a)));
    const int grid = A.items < gpt2_num_sms() ? A.items : gpt2_num_sms();
    if (!A.plan) {
        packed_fwd_tc_kernel<<<grid, THREADS, SMEM, s>>>(mq, mk, mv, A);
        return 1;
    }
    packed_plan_kernel<<<1, 1024, 0, s>>>(a, A.cut, plan);
    if (launch_dependent(packed_fwd_tc_kernel, grid, THREADS, SMEM, s, mq, mk, mv, A) != cudaSuccess)
        return GPT2_ERR_CUDA;
    return 2;
}
