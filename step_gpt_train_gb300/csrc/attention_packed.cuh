// What the kernels of attention over packed sequences share: finding the
// sequence of a row or work item, with offsets that may be out of order.
#pragma once

#include "common.cuh"
#include "launch.h"

#define GPT2_FLAG_OFFSETS 8

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

// A work item of the query-tile kernels: `per` consecutive queries of one
// sequence (less at its end).
struct PackedTile {
    int q0, nq;   // first row in the buffer, queries
    int k0, lk;   // the sequence's keys
    int vis;      // keys that the first query sees (may be negative)
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
int launch_packed_plan(const PackedAttn& a, PackedPlan* plan, int per, cudaStream_t s);

__device__ __forceinline__ PackedTile packed_tile(const PackedSeq& p, int at, int per) {
    PackedTile t = {p.q0 + at, min(per, p.lq - at), p.k0, p.lk, at + 1 + p.lk - p.lq, {0, 0, 0}};
    return t;
}
// Key blocks of 128 that the first n queries of a tile see.
__device__ __forceinline__ int packed_blocks(const PackedTile& t, int n) {
    return n > 0 ? (max(0, t.vis + n - 1) + 127) / 128 : 0;
}
