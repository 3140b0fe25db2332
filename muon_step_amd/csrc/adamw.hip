// AdamW over many tensors in mixed types, moments in 32 bits (adamw_mixed_kernel)
// or in 8 (adamw8_kernel).  Embedding and head tensors, norms, biases and gates
// take AdamW (the deep-dive page, "为什么嵌入层、输出头、bias、RMSNorm 还在用 AdamW").
//
// Compiled with -ffp-contract=off: a multiply and an add round once each unless
// the code says fma.
//
// Both kernels are bound by HBM.  The 32-bit step moves every byte once (by
// counter 2.94 GB each way for its 28 bytes an element on 210e6 elements).  The
// 8-bit step needs 1.27 GB in and 0.85 out for bf16 weights and gradients, 10.1
// bytes an element, and by counter fetches 1.36 and writes 0.87: lines of scales
// that workgroups on several XCDs share.  A plain copy moves 6.4 TB/s on the same
// card; 210e6 elements take
//   32-bit moments, bf16 weights + fp32 master, bf16 gradients   932 us  6.3 TB/s
//   8-bit moments, bf16 weights and gradients                    328 us  6.5 TB/s
//   8-bit moments, bf16 weights + fp32 master, fp32 gradients    607 us  6.3 TB/s
// One vector a lane and one wave a workgroup: in workgroups of 128, 256 and 512
// threads the first takes 946, 983 and 1018 us (smaller calls the same), with
// two or four vectors a lane (256 threads) 1056 and 1018.
#include <algorithm>

#include "adamw_math.hpp"
#include "kernels.hpp"
#include "tensor_table.hpp"
#include "vector_access.hpp"

namespace muon {

namespace {

constexpr int kThreads = 64;  // one wave: see above

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

// Every tensor is read and written once: all accesses are non-temporal.  Where
// the caches hold other data, as after a model's backward pass, that is what
// counts: 128 MB take 27.6 us (32 MB 9.9, 1 GB 173; plain loads 32.0, 13.4 and
// 193, plain stores 28.0, 10.7 and 186).  Only calls of some 64 to 128 MB in a
// loop, which the Infinity Cache could hold, would gain from plain loads (128
// MB 24.2 to 21.3 us).
//
// PACED (calls that move more than 512 MB): each tensor's load is waited for
// before the next tensor's is issued.  With all of a lane's loads in flight on
// every CU the HBM serves five to seven streams at once and gets slower: the
// first of the steps above takes 931 us paced and 958 not, the second 327 and
// 336; calls of 256 MB and less gain nothing.
template <bool PACED> __device__ __forceinline__ void pace() {
    if constexpr (PACED) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// V consecutive values as floats, in 16-byte accesses (8-byte ones for four
// bf16).
template <int V> __device__ __forceinline__ void load_vec(const float *p, float (&x)[V]) {
    static_assert(V == 4, "one access");
    uint32_t w[4];
    load_words<4, 4>(p, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
}
template <int V> __device__ __forceinline__ void load_vec(const uint16_t *p, float (&x)[V]) {
    uint32_t w[V / 2];
    load_words<V / 2, 2>(p, w);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <int V> __device__ __forceinline__ void store_vec(float *p, const float (&x)[V]) {
    static_assert(V == 4, "one access");
    const uint32_t w[4] = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
    store_words<4, 4>(p, w);
}
template <int V> __device__ __forceinline__ void store_vec(uint16_t *p, const float (&x)[V]) {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    store_words<V / 2, 2>(p, w);
}

// The first n of V values (a tensor's last ones), the others zero.
template <int V, class T> __device__ __forceinline__ void load_first(const T *p, int n, float (&x)[V]) {
#pragma unroll
    for (int q = 0; q < V; ++q) x[q] = q < n ? load_one(p + q) : 0.0f;
}
template <int V, class T> __device__ __forceinline__ void store_first(T *p, int n, const float (&x)[V]) {
#pragma unroll
    for (int q = 0; q < V; ++q)
        if (q < n) store_one(p + q, x[q]);
}

// Multiplies by the clip factor (one rounding), when the call has one.
template <int V> __device__ __forceinline__ void clip(const float *factor, float (&g)[V]) {
    if (!factor) return;
    const float f = *as_global(factor);
#pragma unroll
    for (int q = 0; q < V; ++q) g[q] = f * g[q];
}

// ---------------------------------------------------------------------------
// Moments in 32 bits.  Per element the fp32 operations of muon_adamw_step in
// their order, each rounded once (division and square root correctly).  Some 80
// vector instructions an element for that hide behind the memory: with
// approximate division and root a call of 92 MB takes 17.4 us instead of 18.2,
// one of 5.9 GB the same.
constexpr int kMixedVec = 4;                       // elements of a lane
constexpr int kMixedBlock = kThreads * kMixedVec;  // elements of a workgroup

template <int V>
__device__ __forceinline__ void adamw_exact(const AdamwScalars &k, float (&p)[V], const float (&g)[V], float (&m)[V],
                                            float (&v)[V]) {
#pragma unroll
    for (int q = 0; q < V; ++q) {
        const float p1 = k.decay * p[q];
        m[q] = k.beta1 * m[q] + k.one_minus_beta1 * g[q];
        v[q] = k.beta2 * v[q] + (k.one_minus_beta2 * g[q]) * g[q];
        const float den = sqrt_rn(__fdiv_rn(v[q], k.bias_corr2)) + k.eps;
        p[q] = p1 - k.lr * __fdiv_rn(__fdiv_rn(m[q], k.bias_corr1), den);
    }
}

template <typename ParamT, typename GradT, bool MASTER, bool PACED>
__global__ __launch_bounds__(kThreads) void adamw_mixed_kernel(const MixedTable t, uint32_t block0, AdamwScalars k,
                                                               const float *factor) {
    constexpr int V = kMixedVec;
    const uint32_t b = block0 + blockIdx.x;
    const int e = Owners<64>(t.first).of(b);
    const MixedDesc d = t.d[e];
    const int64_t k0 = static_cast<int64_t>(b - t.first[e]) * kMixedBlock;
    ParamT *param = static_cast<ParamT *>(d.param) + k0;
    const GradT *grad = static_cast<const GradT *>(d.grad) + k0;
    float *master = MASTER ? d.master + k0 : nullptr, *dm = d.m + k0, *dv = d.v + k0;
    const int i = threadIdx.x * V;
    const int n = static_cast<int>(min<int64_t>(d.numel - k0, kMixedBlock)) - i;  // elements from this lane's first on
    float p[V], g[V], m[V], v[V];
    if (n >= V) {
        if constexpr (MASTER)
            load_vec(master + i, p);
        else
            load_vec(param + i, p);
        pace<PACED>();
        load_vec(grad + i, g);
        pace<PACED>();
        load_vec(dm + i, m);
        pace<PACED>();
        load_vec(dv + i, v);
    } else {
        if constexpr (MASTER)
            load_first(master + i, n, p);
        else
            load_first(param + i, n, p);
        load_first(grad + i, n, g);
        load_first(dm + i, n, m);
        load_first(dv + i, n, v);
    }
    clip(factor, g);
    adamw_exact(k, p, g, m, v);
    if (n >= V) {
        store_vec(dm + i, m);
        store_vec(dv + i, v);
        if constexpr (MASTER) store_vec(master + i, p);
        store_vec(param + i, p);
    } else {
        store_first(dm + i, n, m);
        store_first(dv + i, n, v);
        if constexpr (MASTER) store_first(master + i, n, p);
        store_first(param + i, n, p);
    }
}

// ---------------------------------------------------------------------------
// Moments in 8 bits: e4m3 codes with an e8m0 scale for each 32 elements, which
// four (eight) neighbouring lanes of eight (four) elements hold.  The moments'
// new values are fp32 with each operation rounded once, so that the codes are
// defined bit for bit; the weights are computed from those values (not from
// their codes) in fp32 with the hardware's square root and reciprocal: the
// correctly rounded ones would take more time than the 10 bytes an element.
//
// Rounding is stochastic: with three mantissa bits a moving average rounded to
// nearest stops moving (0.95 x 1.125 rounds back to 1.125), while the expected
// value of the code here is the value itself.  v_cvt_sr_fp8_f32 rounds up where
// the 20 bits of an fp32 significand that are cut off and the random operand's
// top 20 bits carry.  One hash serves four elements, turned by a byte for each
// and by two more for the second moment: each of its bytes leads one rounding of
// either moment.

// A 32-bit mixing function: two rounds of xor-shift and multiplication.
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    return x ^ (x >> 16);
}

// The largest value of the lanes that share a block of 32 elements: 32 / V
// neighbours (DPP: within quads, then between the two quads of eight lanes).
template <int V> __device__ __forceinline__ uint32_t block_max(uint32_t x) {
    auto with = [](uint32_t a, int b) { return max(a, static_cast<uint32_t>(b)); };
    x = with(x, __builtin_amdgcn_mov_dpp(static_cast<int>(x), 0xB1, 0xf, 0xf, true));             // lane ^ 1
    x = with(x, __builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x4E, 0xf, 0xf, true));             // lane ^ 2
    if (V == 4) x = with(x, __builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x141, 0xf, 0xf, true));  // 7 - lane of 8
    return x;
}

// The value of an e8m0 byte: 2^(e - 127), NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t e) {
    return e == 255 ? __builtin_nanf("") : __uint_as_float(max(e << 23, 0x00400000u));
}

template <int V> __device__ __forceinline__ void decode(const uint32_t (&w)[V / 4], float scale, float (&x)[V]) {
    typedef float floatx2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
        const floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[h]), false);
        const floatx2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[h]), true);
        x[4 * h] = scale * a[0];
        x[4 * h + 1] = scale * a[1];
        x[4 * h + 2] = scale * b[0];
        x[4 * h + 3] = scale * b[1];
    }
}

// V values of a block to codes.  The scale exponent e is the smallest that
// brings the block's largest magnitude to 448 or less (to (224, 448], the upper
// end of e4m3), 17 at least; the product with 2^(127 - e) is exact.  FLOOR: no
// value of a block that holds anything but zeros is coded below 2^-9, the
// smallest code above zero.  A block that holds an infinity or a NaN becomes
// NaN throughout (e = 255).  hashed: the random word of each group of
// four; element j of a group takes it turned left by 8 j + TURN.
template <bool FLOOR, int TURN, int V>
__device__ __forceinline__ void encode(const float (&x)[V], const uint32_t (&hashed)[V / 4], uint32_t (&w)[V / 4],
                                       uint32_t &e_out) {
    uint32_t a = 0;  // as bit patterns NaN is above infinity, and infinity above every finite value
#pragma unroll
    for (int q = 0; q < V; ++q) a = max(a, __float_as_uint(x[q]) & 0x7fffffffu);
    a = block_max<V>(a);
    const bool bad = a >= 0x7f800000u;
    const uint32_t e = max((a + 0x1fffffu) >> 23, 25u) - 8u;
    const float nan = __builtin_nanf("");
    const float inv = bad ? nan : __uint_as_float((254u - e) << 23);
    const float least = bad ? nan : (a != 0 ? 0x1p-9f : 0.0f);
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
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
    e_out = bad ? 255u : e;
}

// Elements of a lane: 16 bytes of the widest tensor, so that a wave's load of
// it is contiguous (eight elements of fp32 in two loads of every other 16 bytes
// each: 5.4 instead of 5.9 TB/s with fp32 master weights and gradients; four
// elements of bf16 in 8-byte loads: 6.0 instead of 6.3 TB/s).
template <typename ParamT, typename GradT, bool MASTER> constexpr int byte_vec() {
    return sizeof(ParamT) == 2 && sizeof(GradT) == 2 && !MASTER ? 8 : 4;
}

// What a lane holds of one vector: V elements and their block's scales.
template <int V> struct ByteLane {
    float p[V], g[V];
    uint32_t m[V / 4], v[V / 4];  // codes
    uint32_t m_scale, v_scale;
};

// The codes of V elements, or of the first n of them.
template <int V> __device__ __forceinline__ void load_first_codes(const uint8_t *p, int n, uint32_t (&w)[V / 4]) {
#pragma unroll
    for (int h = 0; h < V / 4; ++h) w[h] = 0u;
#pragma unroll
    for (int q = 0; q < V; ++q)
        if (q < n) w[q >> 2] |= static_cast<uint32_t>(*as_global(p + q)) << (8 * (q & 3));
}
template <int V> __device__ __forceinline__ void store_first_codes(uint8_t *p, int n, const uint32_t (&w)[V / 4]) {
#pragma unroll
    for (int q = 0; q < V; ++q)
        if (q < n) *as_global(p + q) = static_cast<uint8_t>(w[q >> 2] >> (8 * (q & 3)));
}

constexpr float kSmallEps = 0x1p-38f;

// sqrt(v / (1 - b2^step)) + eps.  v_sqrt_f32 takes subnormal values, whose roots
// are below 2^-63, for zero: against kSmallEps that is less than 2^-25 of
// the sum.  SMALL_EPS: under a smaller eps values below 2^-96 are lifted by 2^32.
// It has kernels of its own: a branch on eps in one kernel costs bf16 weights and
// gradients 1 to 2% (210e6 elements 328 to 331 and 335 us, by how it is placed).
template <bool SMALL_EPS> __device__ __forceinline__ float denominator(const Adamw8Scalars &k, float v) {
    if constexpr (!SMALL_EPS) return __builtin_amdgcn_sqrtf(v * k.inv_bias_corr2) + k.eps;
    const bool low = v < 0x1p-96f;
    const float root = __builtin_amdgcn_sqrtf(v * (low ? 0x1p32f * k.inv_bias_corr2 : k.inv_bias_corr2));
    return __builtin_fmaf(root, low ? 0x1p-16f : 1.0f, k.eps);
}

// The step on the V elements from `i0` of their tensor on.
template <int V, bool SMALL_EPS>
__device__ __forceinline__ void adamw8_lane(const Adamw8Scalars &k, const float *factor, int64_t i0, ByteLane<V> &x) {
    float m[V], v[V];
    decode<V>(x.m, scale_value(x.m_scale), m);
    decode<V>(x.v, scale_value(x.v_scale), v);
    clip(factor, x.g);
#pragma unroll
    for (int q = 0; q < V; ++q) {
        m[q] = k.beta1 * m[q] + k.one_minus_beta1 * x.g[q];
        v[q] = k.beta2 * v[q] + (k.one_minus_beta2 * x.g[q]) * x.g[q];
        const float den = denominator<SMALL_EPS>(k, v[q]);
        // the moment comes in last: neither product leaves fp32's range before the result does
        x.p[q] = __builtin_fmaf(-k.lr_over_bias_corr1 * __builtin_amdgcn_rcpf(den), m[q], k.decay * x.p[q]);
    }
    const uint64_t group = static_cast<uint64_t>(i0) >> 2;
    const uint32_t key = k.key ^ (static_cast<uint32_t>(group >> 32) * 0x9E3779B9u);
    uint32_t hashed[V / 4];
#pragma unroll
    for (int h = 0; h < V / 4; ++h) hashed[h] = mix32((static_cast<uint32_t>(group) + h) ^ key);
    encode<false, 0>(m, hashed, x.m, x.m_scale);
    encode<true, 16>(v, hashed, x.v, x.v_scale);
}

template <typename ParamT, typename GradT, bool MASTER, bool PACED, bool SMALL_EPS>
__global__ __launch_bounds__(kThreads) void adamw8_kernel(const ByteTable t, uint32_t block0, Adamw8Scalars k,
                                                          const float *factor) {
    constexpr int V = byte_vec<ParamT, GradT, MASTER>();
    constexpr int kBlock = kThreads * V;
    const uint32_t b = block0 + blockIdx.x;
    const int e = Owners<64>(t.first).of(b);
    const ByteDesc d = t.d[e];
    const int64_t k0 = static_cast<int64_t>(b - t.first[e]) * kBlock;
    ParamT *param = static_cast<ParamT *>(d.param) + k0;
    const GradT *grad = static_cast<const GradT *>(d.grad) + k0;
    float *master = MASTER ? d.master + k0 : nullptr;
    uint8_t *dm = d.m + k0, *dv = d.v + k0, *ms = d.m_scale + (k0 >> 5), *vs = d.v_scale + (k0 >> 5);
    const int i = threadIdx.x * V;
    // Elements from this lane's first on.  Lanes past the end stay for the
    // reduction over their block: they hold zeros and store nothing.
    const int n = static_cast<int>(min<int64_t>(d.numel - k0, kBlock)) - i;
    ByteLane<V> x;
    x.m_scale = n > 0 ? *as_global(ms + (i >> 5)) : 0u;
    x.v_scale = n > 0 ? *as_global(vs + (i >> 5)) : 0u;
    if (n >= V) {
        if constexpr (MASTER)
            load_vec(master + i, x.p);
        else
            load_vec(param + i, x.p);
        pace<PACED>();
        load_vec(grad + i, x.g);
        pace<PACED>();
        load_words<V / 4, 1>(dm + i, x.m);
        pace<PACED>();
        load_words<V / 4, 1>(dv + i, x.v);
    } else {
        if constexpr (MASTER)
            load_first(master + i, n, x.p);
        else
            load_first(param + i, n, x.p);
        load_first(grad + i, n, x.g);
        load_first_codes<V>(dm + i, n, x.m);
        load_first_codes<V>(dv + i, n, x.v);
    }
    adamw8_lane<V, SMALL_EPS>(k, factor, k0 + i, x);
    if (n >= V) {
        store_words<V / 4, 1>(dm + i, x.m);
        store_words<V / 4, 1>(dv + i, x.v);
        if constexpr (MASTER) store_vec(master + i, x.p);
        store_vec(param + i, x.p);
    } else {
        store_first_codes<V>(dm + i, n, x.m);
        store_first_codes<V>(dv + i, n, x.v);
        if constexpr (MASTER) store_first(master + i, n, x.p);
        store_first(param + i, n, x.p);
    }
    if (n > 0 && (i & 31) == 0) {
        *as_global(ms + (i >> 5)) = static_cast<uint8_t>(x.m_scale);
        *as_global(vs + (i >> 5)) = static_cast<uint8_t>(x.v_scale);
    }
}

// The grid of one launch: a launch's work items are counted in 32 bits.
constexpr uint32_t kMaxGrid = 1u << 23;

template <class Table, class Scalars, class Kernel>
hipError_t launch_table(Kernel kernel, const Table &t, uint32_t blocks, const Scalars &k, const float *factor,
                        hipStream_t st) {
    static_assert(sizeof(Table) <= kTableBytes && sizeof(Table) + sizeof(Scalars) + 16 <= 4096, "kernel arguments");
    for (uint32_t b0 = 0; b0 < blocks; b0 += kMaxGrid) {
        hipLaunchKernelGGL(kernel, dim3(std::min(kMaxGrid, blocks - b0)), dim3(kThreads), 0, st, t, b0, k, factor);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace

int64_t adamw_mixed_blocks(int64_t numel, const AdamwTypes &) { return (numel + kMixedBlock - 1) / kMixedBlock; }
int64_t adamw8_blocks(int64_t numel, const AdamwTypes &y) {
    const int block = kThreads * (y.param_bf16 && y.grad_bf16 && !y.master ? byte_vec<uint16_t, uint16_t, false>()
                                                                           : byte_vec<float, float, false>());
    return (numel + block - 1) / block;
}

namespace {

template <bool PACED>
hipError_t launch_mixed(const MixedTable &t, uint32_t blocks, const AdamwTypes &y, const AdamwScalars &k,
                        const float *factor, hipStream_t st) {
    if (!y.param_bf16)
        return y.grad_bf16 ? launch_table(adamw_mixed_kernel<float, uint16_t, false, PACED>, t, blocks, k, factor, st)
                           : launch_table(adamw_mixed_kernel<float, float, false, PACED>, t, blocks, k, factor, st);
    if (y.master)
        return y.grad_bf16 ? launch_table(adamw_mixed_kernel<uint16_t, uint16_t, true, PACED>, t, blocks, k, factor, st)
                           : launch_table(adamw_mixed_kernel<uint16_t, float, true, PACED>, t, blocks, k, factor, st);
    return y.grad_bf16 ? launch_table(adamw_mixed_kernel<uint16_t, uint16_t, false, PACED>, t, blocks, k, factor, st)
                       : launch_table(adamw_mixed_kernel<uint16_t, float, false, PACED>, t, blocks, k, factor, st);
}

template <bool PACED, bool SMALL_EPS>
hipError_t launch_bytes(const ByteTable &t, uint32_t blocks, const AdamwTypes &y, const Adamw8Scalars &k,
                        const float *factor, hipStream_t st) {
    if (!y.param_bf16)
        return y.grad_bf16 ? launch_table(adamw8_kernel<float, uint16_t, false, PACED, SMALL_EPS>, t, blocks, k, factor, st)
                           : launch_table(adamw8_kernel<float, float, false, PACED, SMALL_EPS>, t, blocks, k, factor, st);
    if (y.master)
        return y.grad_bf16 ? launch_table(adamw8_kernel<uint16_t, uint16_t, true, PACED, SMALL_EPS>, t, blocks, k, factor, st)
                           : launch_table(adamw8_kernel<uint16_t, float, true, PACED, SMALL_EPS>, t, blocks, k, factor, st);
    return y.grad_bf16 ? launch_table(adamw8_kernel<uint16_t, uint16_t, false, PACED, SMALL_EPS>, t, blocks, k, factor, st)
                       : launch_table(adamw8_kernel<uint16_t, float, false, PACED, SMALL_EPS>, t, blocks, k, factor, st);
}

}  // namespace

hipError_t launch_adamw_mixed(const MixedTable &t, uint32_t blocks, const AdamwTypes &y, bool paced,
                              const AdamwScalars &k, const float *factor, hipStream_t st) {
    return paced ? launch_mixed<true>(t, blocks, y, k, factor, st) : launch_mixed<false>(t, blocks, y, k, factor, st);
}

hipError_t launch_adamw8(const ByteTable &t, uint32_t blocks, const AdamwTypes &y, bool paced, const Adamw8Scalars &k,
                         const float *factor, hipStream_t st) {
    if (k.eps < kSmallEps)
        return paced ? launch_bytes<true, true>(t, blocks, y, k, factor, st)
                     : launch_bytes<false, true>(t, blocks, y, k, factor, st);
    return paced ? launch_bytes<true, false>(t, blocks, y, k, factor, st)
                 : launch_bytes<false, false>(t, blocks, y, k, factor, st);
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
