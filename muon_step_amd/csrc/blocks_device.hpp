// Device code that the kernels of the block step share (see blocks.hpp for the method).
#pragma once

#include <type_traits>

#include "blocks.hpp"
#include "tensor_table.hpp"

namespace muon {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;  // of a streaming workgroup (sum_tile adds up as many)
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

// x = hi + lo to 2^-24 of x, each part rounded to nearest (two values an instruction),
// |x| below 65504; parts below 2^-25 are lost.  Truncated parts (2% faster in the
// chain) err to one side, and what lo lo leaves out adds up: O is 3e-6 off on even
// spectra instead of 1e-6.
// HI: which parts the compiler has to hold as two to a register from the conversion
// on.  Left to itself, or told of the others, it spills 53 to 74 registers in the chain
// (HI) and up to 29 in X X^T (low parts; 128 blocks of 128 x 4096 568 us instead of 558).
template <bool HI> __device__ __forceinline__ void split_half(const float (&x)[8], half8 &hi, half8 &lo) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        uint32_t h = __builtin_bit_cast(uint32_t, half2_t{static_cast<_Float16>(x[k]), static_cast<_Float16>(x[k + 1])});
        if constexpr (HI) asm("" : "+v"(h));
        // x - hi, with the conversion of hi in the same instruction
        float d0, d1;
        asm("v_fma_mix_f32 %0, -%1, 1.0, %2 op_sel_hi:[1,0,0]" : "=v"(d0) : "v"(h), "v"(x[k]));
        asm("v_fma_mix_f32 %0, -%1, 1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(d1) : "v"(h), "v"(x[k + 1]));
        uint32_t lw = __builtin_bit_cast(uint32_t, half2_t{static_cast<_Float16>(d0), static_cast<_Float16>(d1)});
        if constexpr (!HI) asm("" : "+v"(lw));
        const half2_t hh = __builtin_bit_cast(half2_t, h), l = __builtin_bit_cast(half2_t, lw);
        hi[k] = hh[0];
        hi[k + 1] = hh[1];
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

// Scales of the fp16 pairs of A and Q: |A| <= 16, |Q| <= 60 and |A Q| <= 60 in the
// schedules that the host admits, so A Q's product of scales, 1024, keeps it below
// 65504 too, and |A| >= 2^-9 (blocks_plan.hpp).  P has no such bounds.
constexpr int kLogScaleQ = 4;
constexpr float kScaleA = 64.0f, kScaleQ = 1 << kLogScaleQ;

// The rows 32 wave .. 32 wave + 31 of a block's P as operand fragments, hi and lo.
template <int T>
__device__ __forceinline__ void store_poly(_Float16 *poly, int64_t block, const float (&rows)[32 * T][32 * T + 4], int wave,
                                           int lane) {
    half8 *frag = reinterpret_cast<half8 *>(poly) + block * (T * T * 256);
    const int h = lane >> 5;
#pragma unroll
    for (int k = 0; k < 2 * T; ++k) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = rows[32 * wave + (lane & 31)][16 * k + 8 * (e >> 2) + 4 * h + (e & 3)];
        half8 hi, lo;
        split_half<true>(x, hi, lo);
        frag[(wave * 2 * T + k) * 64 + lane] = hi;
        frag[T * T * 128 + (wave * 2 * T + k) * 64 + lane] = lo;
    }
}

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

// A value at a uniform address and a lane's bytes behind it.
template <class W> __device__ __forceinline__ W load_at(const char *row, uint32_t lane) {
    return *(const W __attribute__((address_space(1))) *)((const char __attribute__((address_space(1))) *)row + lane);
}
template <class W> __device__ __forceinline__ void store_at(char *row, uint32_t lane, const W &v) {
    *(W __attribute__((address_space(1))) *)((char __attribute__((address_space(1))) *)row + lane) = v;
}
// N words at an address that A divides.
template <int N, int A> struct WordsAt {
    typedef uint32_t type __attribute__((ext_vector_type(N), aligned(A)));
};

// Sum of a tile over the waves of a workgroup to dst, as its lanes hold it (four
// rows of a column a lane: register 4 q + e of lane i at 256 q + 4 i + e).  k
// alternates between two buffers of sh (4 KB for each wave each), so that one
// barrier a tile suffices.
__device__ __forceinline__ void sum_tile(float *dst, float *sh, int k, const floatx16 &tile) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    float *buf = sh + (k & 1) * kWaves * 1024;
#pragma unroll
    for (int r = 0; r < 16; ++r) buf[wave * 1024 + r * 64 + lane] = tile[r];
    __syncthreads();
    floatx4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float *x = buf + (4 * wave + e) * 64 + lane;
        v[e] = x[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v[e] += x[1024 * w];
    }
    *(floatx4 __attribute__((address_space(1))) *)(dst + 256 * wave + 4 * lane) = v;
}

// The lower triangle's 32 x 32 tiles of a sum of X X^T over columns of X, from
// fragments of 32 rows and 16 columns.
template <int T> struct Triangle {
    floatx16 tile[tri(T)];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < tri(T); ++k)
#pragma unroll
            for (int r = 0; r < 16; ++r) tile[k][r] = 0.0f;
    }
    // Adds 16 columns, given as hi and lo fragments of each of X's T row blocks.  The
    // diagonal's lo lo are squares and do not average out, 2^-20 of it in bf16 parts:
    // without them O was 3e-5 to 1e-4 off on spectra over three decades, with them
    // 1e-5 (of fp16 parts they are 2^-24).
    template <class V> __device__ __forceinline__ void add(const V (&hi)[T], const V (&lo)[T]) {
        constexpr int kProducts = std::is_same_v<V, bf16x8> ? 4 : 3;
#pragma unroll
        for (int k = 0; k < kProducts; ++k)
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int j = 0; j <= i; ++j) {
                    floatx16 &t = tile[tri(i) + j];
                    t = mfma(k & 2 ? lo[i] : hi[i], k & 1 ? lo[j] : hi[j], t);
                }
    }
    // The workgroup's sum to dst, tile by tile; entered behind a barrier.
    __device__ __forceinline__ void reduce(float *dst, float *sh) const {
#pragma unroll
        for (int k = 0; k < tri(T); ++k) sum_tile(dst + k * 1024, sh, k, tile[k]);
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
