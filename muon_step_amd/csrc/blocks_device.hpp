// Device code that the kernels of the block step share (see blocks.hpp for the method).
#pragma once

#include <type_traits>

#include "blocks.hpp"
#include "tensor_table.hpp"

namespace muon {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef __fp16 fp16x2_t __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;  // of a streaming workgroup
constexpr int kThreads = kWaves * 64;

constexpr int tri(int t) { return t * (t + 1) / 2; }

__device__ __forceinline__ floatx16 mfma(half8 a, half8 b, floatx16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ floatx16 mfma(bf16x8 a, bf16x8 b, floatx16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// The row of an accumulator's register r in lane half h.
__device__ __forceinline__ int acc_row(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// x = hi + lo to 2^-21 of x (both parts truncated), |x| below 65504; parts below 2^-24 are lost.
__device__ __forceinline__ void split_half(const float (&x)[8], half8 &hi, half8 &lo) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        const half2_t h = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_pkrtz(x[k], x[k + 1]));
        const half2_t l = __builtin_bit_cast(
            half2_t, __builtin_amdgcn_cvt_pkrtz(x[k] - static_cast<float>(h[0]), x[k + 1] - static_cast<float>(h[1])));
        hi[k] = h[0];
        hi[k + 1] = h[1];
        lo[k] = l[0];
        lo[k + 1] = l[1];
    }
}
// x = hi + lo to 2^-17 of x, each part rounded to nearest.
__device__ __forceinline__ void split_bf(const float (&x)[8], bf16x8 &hi, bf16x8 &lo) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        hi[k] = static_cast<__bf16>(x[k]);
        lo[k] = static_cast<__bf16>(x[k] - static_cast<float>(hi[k]));
    }
}

// Scales of the fp16 pairs: A up to 16 (the host admits schedules that keep
// |X| <= 4), Q up to 64, R up to 64 in magnitude.
constexpr float kScaleA = 256.0f, kScaleQ = 16.0f, kScaleR = 256.0f;
// X of the second and later segments' Gram, |X| <= 4.
constexpr float kScaleX = 8192.0f;

// ---------------------------------------------------------------- places in memory

// A block: its addresses, whatever its weight.
struct Place {
    float *mom;
    const char *grad;
    char *param;
    float *out;
    int64_t mom_pitch, grad_pitch, param_pitch, out_pitch;
};
template <int GSIZE, int PSIZE>
__device__ __forceinline__ Place locate(const BlockTable &t, const BlockCall &c, uint32_t block) {
    const Owners<kBlockTensors> owners(t.first);
    const int e = owners.of(block);
    const BlockDesc &d = t.d[e];
    const uint32_t q = block - t.first[e];
    const int64_t row = static_cast<int64_t>(q / d.across) * c.block_rows;
    const int64_t col = static_cast<int64_t>(q % d.across) * c.block_cols;
    Place p;
    p.mom_pitch = d.mom_pitch;
    p.grad_pitch = d.grad_pitch;
    p.param_pitch = d.param_pitch;
    p.out_pitch = d.out_pitch;
    p.mom = d.mom + row * p.mom_pitch + col;
    p.grad = static_cast<const char *>(d.grad) + (row * p.grad_pitch + col) * GSIZE;
    p.param = static_cast<char *>(d.param) + (row * p.param_pitch + col) * PSIZE;
    p.out = d.ns_out ? d.ns_out + row * p.out_pitch + col : nullptr;
    return p;
}

template <bool BF16> __device__ __forceinline__ float load_grad(const char *p, int64_t at) {
    if constexpr (BF16) return bf16_bits_to_float(*as_global(reinterpret_cast<const uint16_t *>(p) + at));
    return *as_global(reinterpret_cast<const float *>(p) + at);
}

// N floats / bf16 values at an address that only their size aligns.
template <int N> struct FloatsAt {
    typedef float type __attribute__((ext_vector_type(N), aligned(4)));
};
template <int N> __device__ __forceinline__ void load_floats(const float *p, float (&x)[N]) {
    static_assert(N == 1 || N == 2 || N == 3 || N % 4 == 0, "whole vectors");
    if constexpr (N == 1) {
        x[0] = *as_global(p);
    } else if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const auto v = *(const typename FloatsAt<4>::type __attribute__((address_space(1))) *)(p + i);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i + k] = v[k];
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = as_global(p)[k];
    }
}
template <int N> __device__ __forceinline__ void store_floats(float *p, const float (&x)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            typename FloatsAt<4>::type v;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = x[i + k];
            *(typename FloatsAt<4>::type __attribute__((address_space(1))) *)(p + i) = v;
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) as_global(p)[k] = x[k];
    }
}
template <int N> struct HalvesAt {
    typedef uint16_t type __attribute__((ext_vector_type(N), aligned(2)));
};
template <bool BF16, int N> __device__ __forceinline__ void load_grads(const char *p, int64_t at, float (&x)[N]) {
    if constexpr (!BF16) {
        load_floats<N>(reinterpret_cast<const float *>(p) + at, x);
    } else if constexpr (N % 8 == 0 || N == 4 || N == 2) {
        constexpr int V = N % 8 == 0 ? 8 : N;
#pragma unroll
        for (int i = 0; i < N; i += V) {
            const auto v = *(const typename HalvesAt<V>::type __attribute__((address_space(1))) *)(
                reinterpret_cast<const uint16_t *>(p) + at + i);
#pragma unroll
            for (int k = 0; k < V; ++k) x[i + k] = bf16_bits_to_float(v[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = load_grad<true>(p, at + k);
    }
}

// The lower triangle's tiles of a sum of X X^T over columns of X.
template <int T> struct Triangle {
    floatx16 tile[tri(T)];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < tri(T); ++k)
#pragma unroll
            for (int r = 0; r < 16; ++r) tile[k][r] = 0.0f;
    }
    // Adds 16 columns, given as hi and lo fragments of each of X's T row blocks.
    template <class V> __device__ __forceinline__ void add(const V (&hi)[T], const V (&lo)[T]) {
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
            for (int j = 0; j <= i; ++j) tile[tri(i) + j] = mfma(hi[i], hi[j], tile[tri(i) + j]);
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
            for (int j = 0; j <= i; ++j) tile[tri(i) + j] = mfma(hi[i], lo[j], tile[tri(i) + j]);
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
            for (int j = 0; j <= i; ++j) tile[tri(i) + j] = mfma(lo[i], hi[j], tile[tri(i) + j]);
    }
    // The workgroup's waves' sum, row-major tile by tile, to dst.  sh: two times
    // 4 KB for each wave; entered behind a barrier.
    __device__ __forceinline__ void reduce(float *dst, float *sh) const {
        const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
        for (int k = 0; k < tri(T); ++k) {
            float *buf = sh + (k & 1) * kWaves * 1024;
#pragma unroll
            for (int r = 0; r < 16; ++r) buf[wave * 1024 + acc_row(r, lane >> 5) * 32 + (lane & 31)] = tile[k][r];
            __syncthreads();
            floatx4 v = *reinterpret_cast<const floatx4 *>(buf + threadIdx.x * 4);
#pragma unroll
            for (int w = 1; w < kWaves; ++w) v += *reinterpret_cast<const floatx4 *>(buf + w * 1024 + threadIdx.x * 4);
            *(floatx4 __attribute__((address_space(1))) *)(dst + k * 1024 + threadIdx.x * 4) = v;
        }
    }
};

// Calls fn with a kernel's T, TALL, gradient type and EVEN (wide blocks: always) as constants.
template <class F> hipError_t choose(int s, bool tall, bool bf16, F fn) {
    auto types = [&](auto t) -> hipError_t {
        constexpr std::true_type yes{};
        constexpr std::false_type no{};
        if (!tall) return bf16 ? fn(t, no, yes, yes) : fn(t, no, no, yes);
        if (s % (4 * t.value) == 0) return bf16 ? fn(t, yes, yes, yes) : fn(t, yes, no, yes);
        return bf16 ? fn(t, yes, yes, no) : fn(t, yes, no, no);
    };
    switch (block_tiles(s)) {
        case 1: return types(std::integral_constant<int, 1>{});
        case 2: return types(std::integral_constant<int, 2>{});
        case 3: return types(std::integral_constant<int, 3>{});
        case 4: return types(std::integral_constant<int, 4>{});
    }
    return hipErrorInvalidValue;
}

}  // namespace muon
