// AdamW over many tensors in mixed types, moments in 32 bits (adamw_mixed_kernel)
// or in 8 (adamw8_kernel).  Embedding and head tensors, norms, biases and gates
// take AdamW (the deep-dive page, "为什么嵌入层、输出头、bias、RMSNorm 还在用 AdamW").
//
// Compiled with -ffp-contract=off: a multiply and an add round once each unless
// the code says fma.
#include <algorithm>

#include "adamw_math.hpp"
#include "kernels.hpp"
#include "tensor_table.hpp"

namespace muon {

namespace {

constexpr int kThreads = 256;

template <typename T> __device__ __forceinline__ float load_one(const T *p);
template <> __device__ __forceinline__ float load_one<float>(const float *p) { return *as_global(p); }
template <> __device__ __forceinline__ float load_one<uint16_t>(const uint16_t *p) {
    return bf16_bits_to_float(*as_global(p));
}
template <typename T> __device__ __forceinline__ void store_one(T *p, float v);
template <> __device__ __forceinline__ void store_one<float>(float *p, float v) { *as_global(p) = v; }
template <> __device__ __forceinline__ void store_one<uint16_t>(uint16_t *p, float v) {
    *as_global(p) = float_to_bf16_bits(v);
}

// V consecutive values as floats, in 16-byte accesses (8-byte ones for four
// bf16), non-temporal: every tensor of the step is read and written once.
template <int V> __device__ __forceinline__ void load_vec(const float *p, float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const floatx4 r = __builtin_nontemporal_load(as_global(reinterpret_cast<const floatx4 *>(p + i)));
#pragma unroll
        for (int q = 0; q < 4; ++q) x[i + q] = r[q];
    }
}
template <int V> __device__ __forceinline__ void load_vec(const uint16_t *p, float (&x)[V]) {
    typedef uint32_t words __attribute__((ext_vector_type(V / 2)));
    const words r = __builtin_nontemporal_load(as_global(reinterpret_cast<const words *>(p)));
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        x[2 * i] = __uint_as_float(r[i] << 16);
        x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
}
template <int V> __device__ __forceinline__ void store_vec(float *p, const float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
        __builtin_nontemporal_store(floatx4{x[i], x[i + 1], x[i + 2], x[i + 3]},
                                    as_global(reinterpret_cast<floatx4 *>(p + i)));
}
template <int V> __device__ __forceinline__ void store_vec(uint16_t *p, const float (&x)[V]) {
    typedef uint32_t words __attribute__((ext_vector_type(V / 2)));
    words r;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    __builtin_nontemporal_store(r, as_global(reinterpret_cast<words *>(p)));
}

// Values i0 .. i0 + V - 1 of a tensor of n: in vectors (`vec`: its address and
// i0 allow it and all of them are inside), or one by one, zero past the end.
template <int V, typename T>
__device__ __forceinline__ void load_some(const T *p, int64_t i0, int64_t n, bool vec, float (&x)[V]) {
    if (vec) {
        load_vec<V>(p + i0, x);
    } else {
#pragma unroll
        for (int q = 0; q < V; ++q) x[q] = i0 + q < n ? load_one<T>(p + i0 + q) : 0.0f;
    }
}
template <int V, typename T>
__device__ __forceinline__ void store_some(T *p, int64_t i0, int64_t n, bool vec, const float (&x)[V]) {
    if (vec) {
        store_vec<V>(p + i0, x);
    } else {
#pragma unroll
        for (int q = 0; q < V; ++q)
            if (i0 + q < n) store_one<T>(p + i0 + q, x[q]);
    }
}

// Multiplies by the clip factor (one rounding), when the call has one.
template <int V> __device__ __forceinline__ void clip(const float *factor, float (&g)[V]) {
    if (!factor) return;
    const float f = *as_global(factor);
#pragma unroll
    for (int q = 0; q < V; ++q) g[q] = f * g[q];
}

// ---------------------------------------------------------------------------
// Moments in 32 bits.  Per element the nine fp32 operations of muon_adamw_step
// in their order, each rounded once (division and square root correctly).
constexpr int kMixedVec = 4;                       // elements of a lane
constexpr int kMixedBlock = kThreads * kMixedVec;  // elements of a workgroup

template <typename ParamT, typename GradT, bool MASTER>
__global__ __launch_bounds__(kThreads) void adamw_mixed_kernel(const MixedTable t, uint32_t block0, AdamwScalars k,
                                                               const float *factor) {
    constexpr int V = kMixedVec;
    const uint32_t b = block0 + blockIdx.x;
    const int e = owner_of(t.first, b);
    const MixedDesc d = t.d[e];
    const int64_t i0 = static_cast<int64_t>(b - t.first[e]) * kMixedBlock + threadIdx.x * V;
    if (i0 >= d.numel) return;
    ParamT *param = static_cast<ParamT *>(d.param);
    const GradT *grad = static_cast<const GradT *>(d.grad);
    const uintptr_t low = reinterpret_cast<uintptr_t>(d.param) | reinterpret_cast<uintptr_t>(d.master) |
                          reinterpret_cast<uintptr_t>(d.grad) | reinterpret_cast<uintptr_t>(d.m) |
                          reinterpret_cast<uintptr_t>(d.v);
    const bool vec = (low & 15) == 0 && i0 + V <= d.numel;
    float p[V], g[V], m[V], v[V];
    if constexpr (MASTER)
        load_some<V>(d.master, i0, d.numel, vec, p);
    else
        load_some<V>(param, i0, d.numel, vec, p);
    load_some<V>(grad, i0, d.numel, vec, g);
    load_some<V>(d.m, i0, d.numel, vec, m);
    load_some<V>(d.v, i0, d.numel, vec, v);
    clip(factor, g);
#pragma unroll
    for (int q = 0; q < V; ++q) {
        const float p1 = k.decay * p[q];
        m[q] = k.beta1 * m[q] + k.one_minus_beta1 * g[q];
        v[q] = k.beta2 * v[q] + (k.one_minus_beta2 * g[q]) * g[q];
        const float den = sqrt_rn(__fdiv_rn(v[q], k.bias_corr2)) + k.eps;
        p[q] = p1 - k.lr * __fdiv_rn(__fdiv_rn(m[q], k.bias_corr1), den);
    }
    store_some<V>(d.m, i0, d.numel, vec, m);
    store_some<V>(d.v, i0, d.numel, vec, v);
    if constexpr (MASTER) store_some<V>(d.master, i0, d.numel, vec, p);
    store_some<V>(param, i0, d.numel, vec, p);
}

// ---------------------------------------------------------------------------
// Moments in 8 bits: e4m3 codes with an e8m0 scale for each 32 elements, which
// four neighbouring lanes of eight elements hold.  The moments' new values are
// fp32 with each operation rounded once, so that the codes are defined bit for
// bit; the weights are computed from those values (not from their codes) in
// fp32 with the hardware's square root and reciprocal.
//
// Rounding is stochastic: with three mantissa bits a moving average rounded to
// nearest stops moving (0.95 x 1.125 rounds back to 1.125), while the expected
// value of the code here is the value itself.  v_cvt_sr_fp8_f32 rounds up where
// the 20 bits of an fp32 significand that are cut off and the random operand's
// top 20 bits carry.
constexpr int kByteVec = 8;
constexpr int kByteBlock = kThreads * kByteVec;

// A 32-bit mixing function: two rounds of xor-shift and multiplication.
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    return x ^ (x >> 16);
}

// The largest of four neighbouring lanes' values (rows of a quad by DPP).
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
    const uint32_t y = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0xB1, 0xf, 0xf, true));
    x = max(x, y);
    const uint32_t z = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x4E, 0xf, 0xf, true));
    return max(x, z);
}

// The value of an e8m0 byte: 2^(e - 127), NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t e) {
    return e == 255 ? __builtin_nanf("") : __uint_as_float(max(e << 23, 0x00400000u));
}

// Eight codes from memory.
__device__ __forceinline__ u32x2 load_codes(const uint8_t *p, int64_t i0, int64_t n, bool vec) {
    if (vec) return __builtin_nontemporal_load(as_global(reinterpret_cast<const u32x2 *>(p + i0)));
    u32x2 w = {0u, 0u};
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (i0 + q < n) w[q >> 2] |= static_cast<uint32_t>(*as_global(p + i0 + q)) << (8 * (q & 3));
    return w;
}
__device__ __forceinline__ void store_codes(uint8_t *p, int64_t i0, int64_t n, bool vec, u32x2 w) {
    if (vec) {
        __builtin_nontemporal_store(w, as_global(reinterpret_cast<u32x2 *>(p + i0)));
        return;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (i0 + q < n) *as_global(p + i0 + q) = static_cast<uint8_t>(w[q >> 2] >> (8 * (q & 3)));
}
__device__ __forceinline__ void decode(u32x2 w, float scale, float (&x)[8]) {
    typedef float floatx2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[h]), false);
        const floatx2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[h]), true);
        x[4 * h] = scale * a[0];
        x[4 * h + 1] = scale * a[1];
        x[4 * h + 2] = scale * b[0];
        x[4 * h + 3] = scale * b[1];
    }
}

// Eight values of a block to codes.  The scale exponent e is the smallest that
// brings the block's largest magnitude to 448 or less (to (224, 448], the upper
// end of e4m3), 17 at least; the product with 2^(127 - e) is exact.  FLOOR: no
// value of a block that holds anything but zeros is coded below 2^-9, the
// smallest code above zero.  A block that holds an infinity or a NaN becomes
// NaN throughout (e = 255).  hashed: the random words of the two groups of
// four; element j of a group takes it turned left by 8 j + TURN.
template <bool FLOOR, int TURN>
__device__ __forceinline__ u32x2 encode(const float (&x)[8], const uint32_t (&hashed)[2], uint32_t *e_out) {
    uint32_t a = 0;  // as bit patterns NaN is above infinity, and infinity above every finite value
#pragma unroll
    for (int q = 0; q < 8; ++q) a = max(a, __float_as_uint(x[q]) & 0x7fffffffu);
    a = quad_max(a);
    const bool bad = a >= 0x7f800000u;
    const uint32_t e = max((a + 0x1fffffu) >> 23, 25u) - 8u;
    const float nan = __builtin_nanf("");
    const float inv = bad ? nan : __uint_as_float((254u - e) << 23);
    const float least = bad ? nan : (a != 0 ? 0x1p-9f : 0.0f);
    u32x2 w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int word = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float y = x[4 * h + j] * inv;
            if (FLOOR) y = __builtin_fmaxf(y, least);
            const int turn = (8 * j + TURN) & 31;
            const uint32_t r = __builtin_rotateleft32(hashed[h], turn);
            switch (j) {  // the byte is an immediate operand
                case 0: word = __builtin_amdgcn_cvt_sr_fp8_f32(y, static_cast<int>(r), word, 0); break;
                case 1: word = __builtin_amdgcn_cvt_sr_fp8_f32(y, static_cast<int>(r), word, 1); break;
                case 2: word = __builtin_amdgcn_cvt_sr_fp8_f32(y, static_cast<int>(r), word, 2); break;
                default: word = __builtin_amdgcn_cvt_sr_fp8_f32(y, static_cast<int>(r), word, 3); break;
            }
        }
        w[h] = static_cast<uint32_t>(word);
    }
    *e_out = bad ? 255u : e;
    return w;
}

template <typename ParamT, typename GradT, bool MASTER>
__global__ __launch_bounds__(kThreads) void adamw8_kernel(const ByteTable t, uint32_t block0, Adamw8Scalars k,
                                                          const float *factor) {
    constexpr int V = kByteVec;
    const uint32_t b = block0 + blockIdx.x;
    const int e = owner_of(t.first, b);
    const ByteDesc d = t.d[e];
    const int64_t i0 = static_cast<int64_t>(b - t.first[e]) * kByteBlock + threadIdx.x * V;
    // Lanes past the tensor's end stay for the reduction over their quad: they
    // hold zeros and store nothing.
    ParamT *param = static_cast<ParamT *>(d.param);
    const GradT *grad = static_cast<const GradT *>(d.grad);
    const uintptr_t low = reinterpret_cast<uintptr_t>(d.param) | reinterpret_cast<uintptr_t>(d.master) |
                          reinterpret_cast<uintptr_t>(d.grad);
    const uintptr_t low8 = reinterpret_cast<uintptr_t>(d.m) | reinterpret_cast<uintptr_t>(d.v);
    const bool vec = (low & 15) == 0 && (low8 & 7) == 0 && i0 + V <= d.numel;
    float p[V], g[V], m[V], v[V];
    if constexpr (MASTER)
        load_some<V>(d.master, i0, d.numel, vec, p);
    else
        load_some<V>(param, i0, d.numel, vec, p);
    load_some<V>(grad, i0, d.numel, vec, g);
    const u32x2 mw = load_codes(d.m, i0, d.numel, vec), vw = load_codes(d.v, i0, d.numel, vec);
    const bool inside = i0 < d.numel;
    const int64_t blk = i0 >> 5;
    const uint32_t me = inside ? *as_global(d.m_scale + blk) : 0u, ve = inside ? *as_global(d.v_scale + blk) : 0u;
    decode(mw, scale_value(me), m);
    decode(vw, scale_value(ve), v);
    clip(factor, g);
#pragma unroll
    for (int q = 0; q < V; ++q) {
        m[q] = k.beta1 * m[q] + k.one_minus_beta1 * g[q];
        v[q] = k.beta2 * v[q] + (k.one_minus_beta2 * g[q]) * g[q];
        // 2^24 v / (1 - b2^step): v_sqrt_f32 takes subnormal values for zero
        const float den = __builtin_fmaf(__builtin_amdgcn_sqrtf(v[q] * k.scaled_inv_bias_corr2), 0x1p-12f, k.eps);
        // the moment comes in last: neither product leaves fp32's range before the result does
        p[q] = __builtin_fmaf(-k.lr_over_bias_corr1 * __builtin_amdgcn_rcpf(den), m[q], k.decay * p[q]);
    }
    const uint64_t group = static_cast<uint64_t>(i0) >> 2;
    const uint32_t key = k.key ^ (static_cast<uint32_t>(group >> 32) * 0x9E3779B9u);
    const uint32_t hashed[2] = {mix32(static_cast<uint32_t>(group) ^ key), mix32(static_cast<uint32_t>(group + 1) ^ key)};
    uint32_t me1, ve1;
    const u32x2 mc = encode<false, 0>(m, hashed, &me1), vc = encode<true, 16>(v, hashed, &ve1);
    if (!inside) return;
    store_codes(d.m, i0, d.numel, vec, mc);
    store_codes(d.v, i0, d.numel, vec, vc);
    if ((threadIdx.x & 3) == 0) {
        *as_global(d.m_scale + blk) = static_cast<uint8_t>(me1);
        *as_global(d.v_scale + blk) = static_cast<uint8_t>(ve1);
    }
    if constexpr (MASTER) store_some<V>(d.master, i0, d.numel, vec, p);
    store_some<V>(param, i0, d.numel, vec, p);
}

// The grid of one launch: a launch's work items are counted in 32 bits.
constexpr uint32_t kMaxGrid = 1u << 23;

template <class Table, class Scalars, class Kernel>
hipError_t launch_table(Kernel kernel, const Table &t, uint32_t blocks, const Scalars &k, const float *factor,
                        hipStream_t st) {
    for (uint32_t b0 = 0; b0 < blocks; b0 += kMaxGrid) {
        hipLaunchKernelGGL(kernel, dim3(std::min(kMaxGrid, blocks - b0)), dim3(kThreads), 0, st, t, b0, k, factor);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace

int64_t adamw_mixed_blocks(int64_t numel) { return (numel + kMixedBlock - 1) / kMixedBlock; }
int64_t adamw8_blocks(int64_t numel) { return (numel + kByteBlock - 1) / kByteBlock; }

hipError_t launch_adamw_mixed(const MixedTable &t, uint32_t blocks, const AdamwTypes &y, const AdamwScalars &k,
                              const float *factor, hipStream_t st) {
    if (!y.param_bf16)
        return y.grad_bf16 ? launch_table(adamw_mixed_kernel<float, uint16_t, false>, t, blocks, k, factor, st)
                           : launch_table(adamw_mixed_kernel<float, float, false>, t, blocks, k, factor, st);
    if (y.master)
        return y.grad_bf16 ? launch_table(adamw_mixed_kernel<uint16_t, uint16_t, true>, t, blocks, k, factor, st)
                           : launch_table(adamw_mixed_kernel<uint16_t, float, true>, t, blocks, k, factor, st);
    return y.grad_bf16 ? launch_table(adamw_mixed_kernel<uint16_t, uint16_t, false>, t, blocks, k, factor, st)
                       : launch_table(adamw_mixed_kernel<uint16_t, float, false>, t, blocks, k, factor, st);
}

hipError_t launch_adamw8(const ByteTable &t, uint32_t blocks, const AdamwTypes &y, const Adamw8Scalars &k,
                         const float *factor, hipStream_t st) {
    if (!y.param_bf16)
        return y.grad_bf16 ? launch_table(adamw8_kernel<float, uint16_t, false>, t, blocks, k, factor, st)
                           : launch_table(adamw8_kernel<float, float, false>, t, blocks, k, factor, st);
    if (y.master)
        return y.grad_bf16 ? launch_table(adamw8_kernel<uint16_t, uint16_t, true>, t, blocks, k, factor, st)
                           : launch_table(adamw8_kernel<uint16_t, float, true>, t, blocks, k, factor, st);
    return y.grad_bf16 ? launch_table(adamw8_kernel<uint16_t, uint16_t, false>, t, blocks, k, factor, st)
                       : launch_table(adamw8_kernel<uint16_t, float, false>, t, blocks, k, factor, st);
}

// The rounding's key for one step: the seed and the step count, mixed.
uint32_t adamw8_key(uint64_t seed, int64_t step) {
    const uint64_t s = static_cast<uint64_t>(step);
    uint32_t x = mix32(static_cast<uint32_t>(s >> 32));
    x = mix32(static_cast<uint32_t>(s) ^ x);
    x = mix32(static_cast<uint32_t>(seed >> 32) ^ x);
    return mix32(static_cast<uint32_t>(seed) ^ x);
}

}  // namespace muon
