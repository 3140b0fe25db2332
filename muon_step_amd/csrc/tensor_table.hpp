// Tables of tensors that travel as kernel arguments.
//
// A launch takes up to N tensors by value in its argument segment (at most
// 4 KB), so a call uploads nothing: it works the same inside a captured graph,
// on any stream, and holds no state between calls.  Tensor k's blocks are
// first[k] .. first[k + 1] - 1; entries past the last tensor hold 0xffffffff.
#pragma once

#include "common.hpp"

namespace muon {

// Finds the tensor that owns a block: the last k with first[k] <= b.  Each lane
// holds N / 64 entries of the table, so the search is one load and N / 64
// ballots instead of a chain of dependent loads.  Uniform over the wave.
template <int N> struct Owners {
    static_assert(N % 64 == 0, "whole waves");
    uint32_t mine[N / 64];
    __device__ __forceinline__ explicit Owners(const uint32_t (&first)[N]) {
#pragma unroll
        for (int i = 0; i < N / 64; ++i) mine[i] = first[i * 64 + (threadIdx.x & 63)];
    }
    __device__ __forceinline__ int of(uint32_t b) const {
        int k = -1;
#pragma unroll
        for (int i = 0; i < N / 64; ++i) k += __popcll(__ballot(mine[i] <= b));
        return __builtin_amdgcn_readfirstlane(k);
    }
};

}  // namespace muon
