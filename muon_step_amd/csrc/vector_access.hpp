// Vector accesses at addresses that their elements alone align.
#pragma once

#include "common.hpp"

namespace muon {

// N words at an address that is a multiple of A bytes only: global memory takes
// vector accesses at any address, so a view that starts anywhere in a flat
// buffer runs as one that is aligned does.
template <int N, int A> struct Words {
    typedef uint32_t type __attribute__((ext_vector_type(N), aligned(A)));
};
template <int N, int A> __device__ __forceinline__ void load_words(const void *p, uint32_t (&w)[N]) {
    typedef const typename Words<N, A>::type __attribute__((address_space(1))) *place;
    const auto r = __builtin_nontemporal_load((place)p);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = r[i];
}
template <int N, int A> __device__ __forceinline__ void store_words(void *p, const uint32_t (&w)[N]) {
    typedef typename Words<N, A>::type vec;
    typedef vec __attribute__((address_space(1))) *place;
    vec r;
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = w[i];
    __builtin_nontemporal_store(r, (place)p);
}

}  // namespace muon
