// What the kernels of attention over packed sequences share: finding the
// sequence of a row or work item, with offsets that may be out of order.
#pragma once

#include "common.cuh"
#include "launch.h"

#define GPT2_FLAG_OFFSETS 8

// SMs of a GB300, where scratch sizes depend on them (they are asked for without a device).
constexpr int PACKED_SMS = 152;

// Launches a kernel that may start while the one before it in the stream still
// runs (its launch and setup hidden behind that), and waits for it itself with
// griddepcontrol.wait before it reads what that kernel wrote.
template <typename... P, typename... V>
inline cudaError_t launch_dependent(void (*kernel)(P...), int grid, int threads, int smem, cudaStream_t s, const V&... v) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, v...);
}

// One sequence's rows: queries q0 .. q0 + lq - 1, keys k0 .. k0 + lk - 1.
// Clamped into the buffers whatever the offsets hold.
struct PackedSeq {
    int q0, lq, k0, lk;
};

__device__ __forceinline__ PackedSeq packed_seq(const PackedAttn& a, int s) {
    PackedSeq p;
    p.q0 = min(max(a.cu_q[s], 0), a.total_q);
    p.lq = min(max(a.cu_q[s + 1], p.q0), a.total_q) - p.q0;
    p.k0 = min(max(a.cu_k[s], 0), a.total_k);
    p.lk = min(max(a.cu_k[s + 1], p.k0), a.total_k) - p.k0;
    return p;
}

// Threads tid, tid + n, ... look their sequences' offsets over: every call
// checks all of them once.
__device__ __forceinline__ void packed_check(const PackedAttn& a, int tid, int n) {
    if (!a.status) return;
    bool bad = false;
    for (int s = tid; s < a.n_seq; s += n) {
        const int q0 = a.cu_q[s], q1 = a.cu_q[s + 1], k0 = a.cu_k[s], k1 = a.cu_k[s + 1];
        bad |= q0 < 0 || q1 < q0 || q1 > a.total_q || q1 - q0 > a.max_q;
        bad |= k0 < 0 || k1 < k0 || k1 > a.total_k || k1 - k0 > a.max_k;
    }
    if (bad) set_status(a.status, GPT2_FLAG_OFFSETS);
}

// The last sequence that starts at or before a row (offsets ascending), or -1.
__device__ __forceinline__ int packed_find_row(const int32_t* cu, int n_seq, int row) {
    int lo = -1, hi = n_seq;  // cu[lo] <= row < cu[hi], with cu[-1] = -inf and cu[n_seq] = inf
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= row) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The work items of a packed batch are tiles of `per` rows of each sequence,
// numbered without a table: sequence s owns the slots floor(cu[s] / per) + s
// up to the next sequence's, which are at least its ceil(len / per) tiles
// (floor(a + len) - floor(a) + 1 >= ceil(len) in units of per) and at most one
// more, so total / per + n_seq slots hold every tile. The last sequence whose
// first slot is at or before `slot`, found by a whole warp (32 probes a
// round), or -1; any offsets give an answer in range.
// (mul: rows to an offset's unit, which `per` counts.)
__device__ __forceinline__ int find_slot(const int32_t* cu, int n_seq, int total, int per, int slot, int& first,
                                         int mul = 1) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n_seq, f_lo = 0;
    bool any = false;
    while (true) {
        const int step = (hi - lo + 31) / 32;
        const int s = lo + lane * step;
        const int f = s < hi ? min(max(cu[s], 0), total) * mul / per + s : 0;
        const uint32_t hit = __ballot_sync(0xffffffffu, s < hi && f <= slot);
        const int c = __popc(hit);
        if (c) {
            any = true;
            f_lo = __shfl_sync(0xffffffffu, f, c - 1);
            lo += (c - 1) * step;
        } else if (!any) {
            return -1;
        }
        if (step == 1) break;
        hi = min(hi, lo + step);
    }
    first = f_lo;
    return lo;
}

// A work item: up to `per` consecutive rows of one sequence, and the rows of
// the other kind that meet them.
//   queries: rows r0 .. r0 + n - 1, keys s0 .. s0 + len - 1 of the sequence;
//     shift = the keys that the first query sees (may be negative);
//   keys: rows r0 .. of keys, queries s0 ..; the first key is seen by the
//     sequence's queries from shift on (may be negative).
struct PackedTile {
    int r0, n;
    int s0, len;
    int shift;
    int pad[3];
};
// The items of a call, the longest first, with a counter from which the CTAs
// of the persistent kernels draw.
struct PackedPlan {
    int next, count, pad[6];
    PackedTile tile[1];
};
inline size_t packed_plan_bytes(int slots) { return 32 + (size_t)slots * sizeof(PackedTile); }
// Slots (at least as many as tiles) of `per` rows: see find_slot.
inline int packed_slots(int total, int n_seq, int per) { return total / per + n_seq; }
constexpr int PACKED_PLAN_MAX = 8192;  // slots that one block sorts in about the time of a launch

// How a kernel cuts its sequences: tiles of `per` queries (or keys), against
// blocks of `block` keys (or queries).
struct PackedCut {
    bool keys;  // the tiles are of keys
    int per, block;
    __host__ __device__ int slots(const PackedAttn& a) const { return (keys ? a.total_k : a.total_q) / per + a.n_seq; }
    __device__ __forceinline__ const int32_t* cu(const PackedAttn& a) const { return keys ? a.cu_k : a.cu_q; }
    __device__ __forceinline__ int total(const PackedAttn& a) const { return keys ? a.total_k : a.total_q; }
    __device__ __forceinline__ int rows(const PackedSeq& p) const { return keys ? p.lk : p.lq; }
    __device__ __forceinline__ PackedTile tile(const PackedSeq& p, int at) const {
        if (keys) return PackedTile{p.k0 + at, min(per, p.lk - at), p.q0, p.lq, at - (p.lk - p.lq), {0, 0, 0}};
        return PackedTile{p.q0 + at, min(per, p.lq - at), p.k0, p.lk, at + 1 + p.lk - p.lq, {0, 0, 0}};
    }
    // Keys: the first of the queries that the blocks cover (a block starts at a multiple of its size).
    __device__ __forceinline__ int first(const PackedTile& t) const { return keys ? max(0, t.shift) / block * block : 0; }
    // Blocks that the tile's first n rows meet.
    __device__ __forceinline__ int blocks(const PackedTile& t, int n) const {
        if (n <= 0) return 0;
        if (keys) return t.shift < t.len ? (t.len - first(t) + block - 1) / block : 0;
        return (max(0, t.shift + n - 1) + block - 1) / block;
    }
};
constexpr int PLAN_SEQ = 2048;  // sequences whose offsets are searched in shared memory
// The tiles of a call sorted by their blocks, most first (a counting sort in
// one block of 1024 threads; equal ones in any order, which changes no result), and the
// counter set to 0. Longest first from one counter leaves the SMs within a
// short item of each other at the end: dealt round robin in sequence order
// they were busy two thirds of the time on 16 ragged prompts.
__device__ __forceinline__ void packed_plan_block(const PackedAttn& a, const PackedCut& cut, PackedPlan* plan,
                                                  bool check) {
    const int slots = cut.slots(a), per = cut.per, total = cut.total(a);
    constexpr int BUCKETS = 1024;
    __shared__ int count[BUCKETS], warps[32], first[PLAN_SEQ], keys[PLAN_SEQ + 1], rows[PLAN_SEQ + 1];
    const int tid = threadIdx.x, lane = tid & 31;
    const bool near = a.n_seq <= PLAN_SEQ;
    if (near)
        for (int s = tid; s <= a.n_seq; s += 1024) {
            rows[s] = a.cu_q[s];
            keys[s] = a.cu_k[s];
            if (s < a.n_seq) first[s] = min(max((cut.keys ? keys : rows)[s], 0), total) / per + s;
        }
    count[tid] = 0;
    __syncthreads();
    PackedAttn c = a;
    if (near) c.cu_q = rows, c.cu_k = keys;
    if (check) packed_check(c, tid, 1024);
    // the tile of a slot, its bucket, or -1
    auto look = [&](int slot, PackedTile& t) -> int {
        int lo = -1, hi = a.n_seq, f = 0;  // the last sequence whose first slot is at or before this one
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            const int x = near ? first[mid] : min(max(cut.cu(a)[mid], 0), total) / per + mid;
            if (x <= slot) lo = mid, f = x;
            else hi = mid;
        }
        if (lo < 0) return -1;
        const PackedSeq p = packed_seq(c, lo);
        const int at = (slot - f) * per;
        if (at < 0 || at >= cut.rows(p)) return -1;
        t = cut.tile(p, at);
        return BUCKETS - 1 - min(cut.blocks(t, t.n), BUCKETS - 1);
    };
    PackedTile t0;
    const int b0 = tid < slots ? look(tid, t0) : -1;
    if (b0 >= 0) atomicAdd(&count[b0], 1);
    for (int slot = tid + 1024; slot < slots; slot += 1024) {
        PackedTile t;
        const int b = look(slot, t);
        if (b >= 0) atomicAdd(&count[b], 1);
    }
    __syncthreads();
    {  // exclusive prefix sums over the buckets
        const int n = count[tid];
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warps[tid >> 5] = x;
        __syncthreads();
        if (tid < 32) {
            int y = warps[tid];
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int z = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) y += z;
            }
            warps[tid] = y;
        }
        __syncthreads();
        x += tid >= 32 ? warps[(tid >> 5) - 1] : 0;
        count[tid] = x - n;
        if (tid == 1023) {
            plan->count = x;
            plan->next = 0;
        }
        __syncthreads();
    }
    if (b0 >= 0) plan->tile[atomicAdd(&count[b0], 1)] = t0;
    for (int slot = tid + 1024; slot < slots; slot += 1024) {
        PackedTile t;
        const int b = look(slot, t);
        if (b >= 0) plan->tile[atomicAdd(&count[b], 1)] = t;
    }
}

