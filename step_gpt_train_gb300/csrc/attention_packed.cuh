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
