// Groups of rows by expert on the device: which expert's rows a work item
// falls on, from the boundary array alone.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace gb300 {

// Where a search for a work item stands: groups before `base` hold `before`
// items (and `blocks` blocks of 128 rows); `start` is group `base`'s first
// row, the running maximum of the boundaries so far.
struct GroupCursor {
    int base = 0;
    int start = 0;
    int before = 0;
    int blocks = 0;
};

struct GroupHit {
    int e;       // the expert
    int start;   // its first row
    int end;     // past its last row
    int local;   // the item's number within the expert
    int block0;  // its first block of 128 rows (rows of every group start a new block)
};

// Boundary i as the kernels take it: clamped to [0, T].
__device__ __forceinline__ int group_bound(const int* offsets, int i, int T) {
    return min(max(__ldg(offsets + i), 0), T);
}

__device__ __forceinline__ GroupCursor group_begin(const int* offsets, int T) {
    GroupCursor c;
    c.start = group_bound(offsets, 0, T);
    return c;
}

// Whole warp.  Finds the group holding item `target` when a group of n rows
// has units(n) items; targets of later calls with the same cursor must not
// decrease.  32 groups a step: a running maximum over the boundaries and a
// running sum over the items, both by shuffles.  False when there are fewer
// than target + 1 items.
template <typename Units>
__device__ __forceinline__ bool group_find(const int* offsets, int E, int T, int target, GroupCursor& c, Units units,
                                           GroupHit& hit) {
    const int lane = threadIdx.x & 31;
    while (c.base < E) {
        const int i = c.base + lane;
        int end = i < E ? group_bound(offsets, i + 1, T) : 0;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, end, d);
            if (lane >= d) end = max(end, v);
        }
        end = max(end, c.start);
        int start = __shfl_up_sync(0xffffffffu, end, 1);
        if (lane == 0) start = c.start;
        const int n = end - start;
        const int u = i < E ? units(n) : 0;
        int items = u, blocks = (n + 127) >> 7;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, items, d);
            const int b = __shfl_up_sync(0xffffffffu, blocks, d);
            if (lane >= d) {
                items += v;
                blocks += b;
            }
        }
        const unsigned int past = __ballot_sync(0xffffffffu, c.before + items > target);
        if (past) {
            const int l = __ffs(past) - 1;
            hit.e = c.base + l;
            hit.start = __shfl_sync(0xffffffffu, start, l);
            hit.end = __shfl_sync(0xffffffffu, end, l);
            hit.local = target - c.before - __shfl_sync(0xffffffffu, items - u, l);
            hit.block0 = c.blocks + __shfl_sync(0xffffffffu, blocks - ((n + 127) >> 7), l);
            return true;
        }
        c.before += __shfl_sync(0xffffffffu, items, 31);
        c.blocks += __shfl_sync(0xffffffffu, blocks, 31);
        c.start = __shfl_sync(0xffffffffu, end, 31);
        c.base += 32;
    }
    return false;
}

// Whole warp.  Items of all groups.
template <typename Units>
__device__ __forceinline__ int group_total(const int* offsets, int E, int T, Units units) {
    const int lane = threadIdx.x & 31;
    int from = group_bound(offsets, 0, T), total = 0;
    for (int base = 0; base < E; base += 32) {
        const int i = base + lane;
        int end = i < E ? group_bound(offsets, i + 1, T) : 0;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, end, d);
            if (lane >= d) end = max(end, v);
        }
        end = max(end, from);
        int start = __shfl_up_sync(0xffffffffu, end, 1);
        if (lane == 0) start = from;
        total += __reduce_add_sync(0xffffffffu, i < E ? units(end - start) : 0);
        from = __shfl_sync(0xffffffffu, end, 31);
    }
    return total;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
    return __float2half_rn(v);
}

// Two of them, the first in the low bits (one instruction).
template <typename T>
__device__ __forceinline__ uint32_t pair_from_f32(float lo, float hi) {
    if constexpr (__is_same(T, __nv_bfloat16)) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

}  // namespace gb300
