// The groups of requests of dattn_decode_shared, as its kernels read them.
#pragma once

#include "common.cuh"

namespace dattn {

// Whether the bounds group_indptr[0 .. groups] ascend within [0, B]; by all nthreads threads of a
// block, one answer.
__device__ __forceinline__ bool shared_groups_ok(const int32_t* indptr, int32_t groups, int32_t B,
                                                 int tid, int nthreads) {
    bool ok = true;
    for (int32_t g = tid; g < groups; g += nthreads) {
        const int32_t a = __ldcg(indptr + g), b = __ldcg(indptr + g + 1);
        ok = ok && a >= 0 && a <= b && b <= B;
    }
    return __syncthreads_and(ok) != 0;
}

// The group of request i, -1 where it is in none; the bounds ascend.
__device__ __forceinline__ int32_t shared_group(const int32_t* indptr, int32_t groups, int32_t i) {
    int32_t lo = 0, hi = groups;  // the number of groups that end at or before i
    while (lo < hi) {
        const int32_t mid = (lo + hi) >> 1;
        if (__ldcg(indptr + mid + 1) <= i) lo = mid + 1; else hi = mid;
    }
    return lo < groups && __ldcg(indptr + lo) <= i ? lo : -1;
}

}  // namespace dattn
