// Tables of tensors that travel as kernel arguments.
//
// A launch takes up to N tensors by value in its argument segment (at most
// 4 KB), so a call uploads nothing: it works the same inside a captured graph,
// on any stream, and holds no state between calls.  Tensor k's blocks are
// first[k] .. first[k + 1] - 1; entries past the last tensor hold 0xffffffff.
#pragma once

#include "common.hpp"

namespace muon {

// The tensor that owns block b: the last k with first[k] <= b.  Each lane
// compares 64 entries of the table at once, so the search is one load and one
// ballot instead of a chain of dependent loads.  Uniform over the wave.
template <int N>
__device__ __forceinline__ int owner_of(const uint32_t (&first)[N], uint32_t b) {
    static_assert(N % 64 == 0, "whole waves");
    int k = -1;
#pragma unroll
    for (int i = 0; i < N / 64; ++i) k += __popcll(__ballot(first[i * 64 + (threadIdx.x & 63)] <= b));
    return __builtin_amdgcn_readfirstlane(k);
}

}  // namespace muon
