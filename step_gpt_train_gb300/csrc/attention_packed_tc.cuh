// What the tcgen05 kernels of packed attention share: tensor maps, the search
// for a work item's sequence, small arithmetic.
#pragma once

#include "attention_packed.cuh"
#include "tc_common.cuh"

namespace packed_tc {

using namespace tc;

constexpr int HD = 64;              // head size
constexpr int TILE = 128 * HD * 2;  // 16 KB: 128 rows of 64 bf16
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// Three-input maximum (one instruction on sm_100 and later).
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// (lo, hi) rounded to a packed bf16 pair, lo in the low half.
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ float f2_total(uint64_t v) {
    float lo, hi;
    f2_unpack(v, lo, hi);
    return lo + hi;
}

// Load 16 consecutive fp32 columns of this thread's TMEM lane (as tc_ld32_issue).
__device__ __forceinline__ void tc_ld16_issue(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tc_ld16_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])
                 :
                 : "memory");
}

// Bounded wait by a whole warp for the phase with the given parity: one try
// and one vote a turn.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
    if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
    const long long t0 = clock64();
    const long long limit = *(volatile long long*)&wait_limit_cycles;
#pragma unroll 1
    for (uint32_t n = 1;; n++) {
        if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
        if (n % 64 == 0) {
            const bool late = clock64() - t0 > limit;
            if (late) {
                set_status(status, GPT2_FLAG_TIMEOUT);
                *abort_flag = 1;
            }
            if (__any_sync(0xffffffffu, late || *abort_flag)) return false;
        }
    }
}

// The next work item of this CTA, by a whole warp: a tile and a key head, from
// the sorted plan or (x counts on from blockIdx.x) from the offsets themselves.
// id (optional): the item's number, from which tile_of finds it again.
__device__ __forceinline__ bool next_tile(const PackedAttn& a, const PackedCut& cut, PackedPlan* plan, int items,
                                          int& x, PackedTile& t, int& kh, int* id = nullptr) {
    if (plan) {
        int n = 0;
        if ((threadIdx.x & 31) == 0) n = atomicAdd(&plan->next, 1);
        n = __shfl_sync(0xffffffffu, n, 0);
        if (n >= plan->count * a.Hkv) return false;
        t = plan->tile[n / a.Hkv];
        kh = n % a.Hkv;
        if (id) *id = n;
        return true;
    }
    const int slots = items / a.Hkv;
    while (x < items) {
        const int i = x;
        x += gridDim.x;
        // the later queries of a sequence, which see more keys, first; the earlier keys, seen by more queries
        const int slot = cut.keys ? i / a.Hkv : slots - 1 - i / a.Hkv;
        int f;
        const int s = find_slot(cut.cu(a), a.n_seq, cut.total(a), cut.per, slot, f);
        if (s < 0) continue;
        const PackedSeq q = packed_seq(a, s);
        const int at = (slot - f) * cut.per;
        if (at < 0 || at >= cut.rows(q)) continue;
        t = cut.tile(q, at);
        kh = i % a.Hkv;
        if (id) *id = i;
        return true;
    }
    return false;
}
// An item that next_tile gave out before.
__device__ __forceinline__ void tile_of(const PackedAttn& a, const PackedCut& cut, const PackedPlan* plan, int items,
                                        int id, PackedTile& t, int& kh) {
    if (plan) {
        t = plan->tile[id / a.Hkv];
        kh = id % a.Hkv;
    } else {
        next_tile(a, cut, nullptr, items, id, t, kh);
    }
}
// Items sorted by length are worth their own launch once there are more than
// SMs to take them; beyond PACKED_PLAN_MAX the sort would cost more than the
// imbalance, which evens out over so many.
inline bool planned(int slots, int Hkv) {
    return (int64_t)slots * Hkv > gpt2_num_sms() && slots <= PACKED_PLAN_MAX;
}

// Rows of [heads][64] bf16 at `stride` elements, viewed as (64, heads, rows)
// with boxes of (64, box_h, box_rows); rows past the end read as zero.
inline bool rows_map(CUtensorMap* map, const void* p, int heads, int rows, int64_t stride, int box_h, int box_rows) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)HD, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)HD * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {HD, (cuuint32_t)box_h, (cuuint32_t)box_rows};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows [from, 128) of a swizzled tile := 0 by one warp, visible to the tensor
// cores before the caller's arrive. (Rows keep their place under the swizzle,
// which only permutes the 16-byte units of a row.)
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int lane) {
    for (int i = from * 8 + lane; i < 128 * 8; i += 32) reinterpret_cast<uint4*>(tile)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
}

}  // namespace packed_tc
