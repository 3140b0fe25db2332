// Muon steps on blocks with a smaller side of at most 128: the heads of an
// attention projection, the factors of an adapter.
//
// X is s x l with s <= 128, so the iteration X <- (a + b A + c A^2) X, A = X X^T,
// need not touch X's long rows at every step: X_k = P_k X_0 with P_k a product
// of s x s polynomials, and A follows in s x s matrices as well,
//     Q = a + b A + c A^2,   A <- Q A Q,   P <- Q P.
// A's rounding noise sits in the directions of small singular values too, where
// each step multiplies it by a^2 (11.9), so A is taken from X = P N again where
// that has grown too far (the host cuts the schedule into segments; the hybrid
// schedule into 4 + 6 steps).  One step over a block then is
//     momentum:  M, N, the partial sums of N N^T                  (reads G, M; writes M)
//     chain:     A = N N^T / ||N||^2, the first segment's P       (s x s, one workgroup a block)
//     regram:    X = P N, the partial sums of X X^T               (reads G, M)
//     chain:     the second segment's P
//     update:    O = P N, W                                       (reads G, M, W; writes W)
// N is formed from M and G wherever it is needed: 6 bytes read an element, where
// a stored X would be 4 written and 4 read.
//
// Products run on the matrix cores with each fp32 operand as a sum of two
// 16-bit parts, hi and lo, and three products hi hi + hi lo + lo hi in fp32
// accumulators: bf16 parts (16 bits of significand) for the first N N^T, whose
// scale is not known before it, fp16 parts (21 bits) of suitably scaled
// matrices everywhere else.
//
// Index basis of the smaller side.  A wave reads 32 lanes x T tiles of it; where
// memory is contiguous along the smaller side (tall blocks, X = N^T) lane i
// takes elements T i .. T i + T - 1, one for each tile, so basis index 32 t + i
// stands for element T i + t; in wide blocks it stands for itself.
//
// Fragments.  v_mfma_f32_32x32x16 wants of either operand, in lane (i, h), i < 32,
// h < 2, eight k of row (column) i; the accumulator holds in lane (j, h) rows
// 8 (r / 4) + 4 h + r % 4, r < 16, of column j.  The order of k is free as long
// as both operands agree, so chunk q (of two) of a tile takes accumulator
// registers 8 q .. 8 q + 7 as they are: an accumulator is the next product's
// operand without leaving its lane.
#include <algorithm>

#include "blocks.hpp"
#include "kernels.hpp"
#include "tensor_table.hpp"

namespace muon {

namespace {

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

// ------------------------------------------------------- momentum, N and N N^T

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

// One part of one block: M <- mu M + G and the sum of N N^T over the part's
// columns.  Outside 2^-40 <= max |N| <= 2^40, where squares could leave fp32's
// range, the part is summed a second time as N 2^-shift.
template <int T, bool TALL, bool BF16>
__global__ __launch_bounds__(kThreads) void blocks_momentum_kernel(const BlockTable t, const BlockCall c) {
    __shared__ __attribute__((aligned(16))) float sh[2 * kWaves * 1024];
    __shared__ uint32_t sh_largest[kWaves];
    const uint32_t block = blockIdx.x / c.parts, part = blockIdx.x % c.parts;  // block: of the launch
    const Place at = locate<BF16 ? 2 : 4, 2>(t, c, c.base + block);
    const int wave = threadIdx.x >> 6, i = threadIdx.x & 31, h = threadIdx.x >> 5 & 1;
    const int begin = part * c.part_len, end = min(begin + c.part_len, c.l);
    const float factor = c.factor ? *c.factor : 1.0f;
    const float mu = c.mu;
    const bool nesterov = c.nesterov != 0;
    uint32_t largest = 0;
    Triangle<T> sum;

    auto note = [&](float n) { largest = max(largest, __float_as_uint(n) & 0x7fffffffu); };

    // 32 columns from x0 on, element by element, past-the-end ones as zeros;
    // again: M is up to date, and N is scaled by 2^-shift.
    auto each = [&](int x0, bool again, int shift) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            bf16x8 hi[T], lo[T];
#pragma unroll
            for (int k = 0; k < T; ++k) {
                const int p = TALL ? T * i + k : 32 * k + i;
                float n[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int x = TALL ? x0 + 16 * q + 8 * h + e : x0 + 16 * h + 8 * q + e;
                    n[e] = 0.0f;
                    if (p < c.s && x < end) {
                        const int64_t row = TALL ? x : p, col = TALL ? p : x;
                        float *m = at.mom + row * at.mom_pitch + col;
                        const float g = load_grad<BF16>(at.grad, row * at.grad_pitch + col) * factor;
                        float v = *as_global(m);
                        if (!again) {
                            v = mu * v + g;
                            *as_global(m) = v;
                        }
                        n[e] = nesterov ? mu * v + g : v;
                    }
                    if (again)
                        n[e] = ldexpf(n[e], -shift);
                    else
                        note(n[e]);
                }
                split_bf(n, hi[k], lo[k]);
            }
            sum.add(hi, lo);
        }
    };
    // 32 columns, all of them inside.
    auto whole = [&](int x0) {
        if constexpr (TALL) {
            const bool mine = T * i < c.s;
            const int p = mine ? T * i : 0;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float m[8][T], g[8][T];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int64_t row = x0 + 16 * q + 8 * h + e;
                    load_floats<T>(at.mom + row * at.mom_pitch + p, m[e]);
                    load_grads<BF16, T>(at.grad, row * at.grad_pitch + p, g[e]);
                }
                bf16x8 hi[T], lo[T];
#pragma unroll
                for (int k = 0; k < T; ++k) {
                    float n[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float gf = g[e][k] * factor;
                        m[e][k] = mu * m[e][k] + gf;
                        n[e] = nesterov ? mu * m[e][k] + gf : m[e][k];
                        n[e] = mine ? n[e] : 0.0f;
                        note(n[e]);
                    }
                    split_bf(n, hi[k], lo[k]);
                }
                if (mine) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        store_floats<T>(at.mom + (x0 + 16 * q + 8 * h + e) * at.mom_pitch + p, m[e]);
                }
                sum.add(hi, lo);
            }
        } else {
            bf16x8 hi[2][T], lo[2][T];
            float m[T][16], g[T][16];
#pragma unroll
            for (int k = 0; k < T; ++k) {
                const int64_t row = min(32 * k + i, c.s - 1);
                load_floats<16>(at.mom + row * at.mom_pitch + x0 + 16 * h, m[k]);
                load_grads<BF16, 16>(at.grad, row * at.grad_pitch + x0 + 16 * h, g[k]);
            }
#pragma unroll
            for (int k = 0; k < T; ++k) {
                const bool mine = 32 * k + i < c.s;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float n[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float gf = g[k][8 * q + e] * factor;
                        float &v = m[k][8 * q + e];
                        v = mu * v + gf;
                        n[e] = nesterov ? mu * v + gf : v;
                        n[e] = mine ? n[e] : 0.0f;
                        note(n[e]);
                    }
                    split_bf(n, hi[q][k], lo[q][k]);
                }
                if (mine) store_floats<16>(at.mom + (32 * k + i) * at.mom_pitch + x0 + 16 * h, m[k]);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) sum.add(hi[q], lo[q]);
        }
    };

    sum.clear();
    const bool vec = !TALL || c.s % T == 0;
    for (int x0 = begin + 32 * wave; x0 < end; x0 += kBlockUnit) {
        if (vec && x0 + 32 <= end)
            whole(x0);
        else
            each(x0, false, 0);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) largest = max(largest, static_cast<uint32_t>(__shfl_xor(static_cast<int>(largest), off, 64)));
    if ((threadIdx.x & 63) == 0) sh_largest[wave] = largest;
    __syncthreads();
    largest = max(max(sh_largest[0], sh_largest[1]), max(sh_largest[2], sh_largest[3]));
    int shift = 0;
    if (largest != 0 && largest < 0x7f800000u) {
        int e;
        (void)frexpf(__uint_as_float(largest), &e);
        if (e < -40 || e > 40) shift = e;
    }
    if (shift != 0) {
        sum.clear();
        for (int x0 = begin + 32 * wave; x0 < end; x0 += kBlockUnit) each(x0, true, shift);
    }
    const int64_t slot = static_cast<int64_t>(block) * c.parts + part;
    sum.reduce(c.w.gram + slot * tri(T) * 1024, sh);
    if (threadIdx.x == 0) c.w.parts[slot] = BlockPart{largest, shift};
}

// ------------------------------------------------------------------- the chain

// s x s matrices, padded with zeros to 32 T; wave w of T holds columns 32 w ..
// 32 w + 31 in accumulator layout.  `left` (shared memory) is a matrix's
// fragments as its columns' waves wrote them, which read as the rows of its
// transpose: a product with it is L^T B.  With A symmetric but for rounding,
//     S = A^T A,  Q = a + b A + c S,  R = A^T Q,  A <- Q^T R,  P <- Q^T P
// keeps A's noise as small as exact transposes would (A <- Q^T Q^T A does not:
// the antisymmetric part of the noise then grows past the rest).
template <int T> struct Slab {
    float v[T][16];
};
template <int T> struct Left {
    half8 hi[T][2 * T][64], lo[T][2 * T][64];
};
template <int T>
__device__ __forceinline__ void put(Left<T> &left, int wave, int lane, const Slab<T> &m, float scale) {
#pragma unroll
    for (int c = 0; c < 2 * T; ++c) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = m.v[c >> 1][8 * (c & 1) + e] * scale;
        half8 hi, lo;
        split_half(x, hi, lo);
        left.hi[wave][c][lane] = hi;
        left.lo[wave][c][lane] = lo;
    }
}
// L^T B, scaled: L was put with its own scale, B is split as B scale, the result multiplied by `out`.
template <int T>
__device__ __forceinline__ Slab<T> product(const Left<T> &left, int lane, const Slab<T> &b, float scale, float out) {
    floatx16 acc[T];
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] = 0.0f;
#pragma unroll
    for (int c = 0; c < 2 * T; ++c) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = b.v[c >> 1][8 * (c & 1) + e] * scale;
        half8 hi, lo;
        split_half(x, hi, lo);
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const half8 ah = left.hi[i][c][lane], al = left.lo[i][c][lane];
            acc[i] = mfma(ah, hi, acc[i]);
            acc[i] = mfma(ah, lo, acc[i]);
            acc[i] = mfma(al, hi, acc[i]);
        }
    }
    Slab<T> r;
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k) r.v[i][k] = acc[i][k] * out;
    return r;
}

// Scales of the fp16 pairs: A up to 16 (the host admits schedules that keep
// |X| <= 4), Q up to 64, R up to 64 in magnitude.
constexpr float kScaleA = 256.0f, kScaleQ = 16.0f, kScaleR = 256.0f;
// X of the second and later segments' Gram, |X| <= 4.
constexpr float kScaleX = 8192.0f;

template <int T> __global__ __launch_bounds__(64 * T, T == 4 ? 2 : 1) void blocks_chain_kernel(const BlockChain c) {
    union Shared {
        Left<T> left;
        float rows[32 * T][32 * T + 4];
    };
    __shared__ __attribute__((aligned(16))) Shared sh;
    __shared__ float sh_sum[T];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, j = lane & 31, h = lane >> 5;
    const int64_t block = blockIdx.x;
    const int col = 32 * wave + j;

    // Sum of a value over the workgroup.
    auto total = [&](float x) {
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off, 64);
        __syncthreads();
        if (lane == 0) sh_sum[wave] = x;
        __syncthreads();
        float r = 0.0f;
#pragma unroll
        for (int w = 0; w < T; ++w) r += sh_sum[w];
        return r;
    };
    // The entries of the diagonal that this lane holds: tile `wave`, its row j.
    auto on_diagonal = [&](int t, int r) { return t == wave && acc_row(r, h) == j; };

    // The parts' common exponent, and what the block holds.
    const BlockPart *parts = c.w.parts + block * c.parts;
    uint32_t largest = 0;
    int common = -1000;
    if (c.first) {
        for (int k = 0; k < c.parts; ++k) {
            largest = max(largest, parts[k].largest);
            if (parts[k].largest != 0) common = max(common, parts[k].shift);
        }
    }
    const bool zero = c.first && largest == 0, bad = c.first && largest >= 0x7f800000u;

    // A: the parts' sum, the upper triangle as the lower one's mirror image.
    Slab<T> a;
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) a.v[t][r] = 0.0f;
    for (int k = 0; k < c.parts; ++k) {
        const float *g = c.w.gram + (block * c.parts + k) * tri(T) * 1024;
        if (c.first && parts[k].largest == 0) continue;
        const float weight = c.first ? ldexpf(1.0f, 2 * (parts[k].shift - common)) : 1.0f;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            if (t >= wave) {
#pragma unroll
                for (int r = 0; r < 16; ++r) a.v[t][r] += weight * g[(tri(t) + wave) * 1024 + acc_row(r, h) * 32 + j];
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const floatx4 v = *reinterpret_cast<const floatx4 *>(g + (tri(wave) + t) * 1024 + j * 32 + 8 * q + 4 * h);
#pragma unroll
                    for (int e = 0; e < 4; ++e) a.v[t][4 * q + e] += weight * v[e];
                }
            }
        }
    }
    if (c.first) {
        float trace = 0.0f;
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) trace += on_diagonal(t, r) ? a.v[t][r] : 0.0f;
        trace = total(trace);
        const double n = sqrt(static_cast<double>(trace));
        const float inv = static_cast<float>(1.0 / (n * n));
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) a.v[t][r] *= inv;
        if (threadIdx.x == 0) {
            int e = 0;  // 2^e <= sqrt(s l) / norm < 2^(e + 1)
            (void)frexp(sqrt(static_cast<double>(c.s) * c.l) / n, &e);
            --e;
            BlockScalars out;
            out.shift = zero || bad ? 0 : e - common;
            out.inv_norm = zero || bad ? 1.0f : static_cast<float>(1.0 / ldexp(n, e));
            out.update = c.update;
            out.pad_ = 0;
            c.w.scalars[block] = out;
        }
    } else {
        constexpr float unscale = 1.0f / (kScaleX * kScaleX);
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) a.v[t][r] *= unscale;
    }

    // P: the identity, or what the segments before made it.
    Slab<T> p;
    float *own = c.w.poly_own + (block * T + wave) * T * 1024;
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            p.v[t][r] = c.first ? (on_diagonal(t, r) ? 1.0f : 0.0f) : own[(t * 16 + r) * 64 + lane];

    Slab<T> q = p;  // the last step's Q, for the norm of what it makes of X
    Slab<T> last_r = a;
    for (int k = 0; k < c.steps; ++k) {
        const BlockChain::Step step = c.step[k];
        put(sh.left, wave, lane, a, kScaleA);
        __syncthreads();
        const Slab<T> s = product(sh.left, lane, a, kScaleA, 1.0f / (kScaleA * kScaleA));
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float diagonal = on_diagonal(t, r) ? step.a : 0.0f;
                q.v[t][r] = diagonal + step.b * a.v[t][r] + step.c * s.v[t][r];
            }
        const bool more = k + 1 < c.steps;
        if (more || (c.last && c.unit_rms)) last_r = product(sh.left, lane, q, kScaleQ, 1.0f / (kScaleA * kScaleQ));
        __syncthreads();
        put(sh.left, wave, lane, q, kScaleQ);
        __syncthreads();
        p = product(sh.left, lane, p, ldexpf(1.0f, -step.exp_in), ldexpf(1.0f / kScaleQ, step.exp_in));
        if (more) a = product(sh.left, lane, last_r, kScaleR, 1.0f / (kScaleQ * kScaleR));
        __syncthreads();
    }

    if (c.last && c.unit_rms) {
        // ||O||^2 = tr Q A Q, or 1 where there was no step
        float sq = 0.0f;
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) sq += q.v[t][r] * last_r.v[t][r];
        sq = total(sq);
        const double o = c.steps > 0 ? sqrt(static_cast<double>(sq)) : 1.0;
        if (threadIdx.x == 0) c.w.scalars[block].update = zero || !(o > 0) ? 0.0f : static_cast<float>(c.update / o);
    }

    // P's columns for the next segment, and its rows as fragments for the products with N.
    const float out = c.steps > 0 ? ldexpf(1.0f, -c.step[c.steps - 1].exp_out) : 1.0f;
    const float nan = __builtin_nanf("");
    __syncthreads();
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float x = zero ? 0.0f : bad ? nan : p.v[t][r];
            if (!c.last) own[(t * 16 + r) * 64 + lane] = x;
            sh.rows[32 * t + acc_row(r, h)][col] = x * out;
        }
    __syncthreads();
    half8 *frag = reinterpret_cast<half8 *>(c.w.poly) + block * (T * T * 256);
#pragma unroll
    for (int k = 0; k < 2 * T; ++k) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = sh.rows[col][16 * k + 8 * (e >> 2) + 4 * h + (e & 3)];
        half8 hi, lo;
        split_half(x, hi, lo);
        frag[(wave * 2 * T + k) * 64 + lane] = hi;
        frag[T * T * 128 + (wave * 2 * T + k) * 64 + lane] = lo;
    }
}

// ------------------------------------------------------------ products with N

// N's values of one lane: of column x, in wide blocks with V columns x .. x + V - 1
// side by side, the entries of basis index 32 t + 16 q + 8 a + 4 h + b.
template <int T, int V> struct Column {
    float n[V][T][2][2][4];  // [column][t][q][a][b]
};

template <bool BF16> __device__ __forceinline__ float nesterov_input(float m, float g, const BlockCall &c, float factor) {
    return c.nesterov ? c.mu * m + g * factor : m;
}

// Wide: columns x0 + V j + v (j the lane), those at or past `end` as zeros.
template <int T, int V, bool BF16, bool TAIL>
__device__ __forceinline__ void load_wide(Column<T, V> &o, const Place &at, const BlockCall &c, float factor, int x0,
                                          int end, int j, int h) {
    float m[T][2][2][4][V], g[T][2][2][4][V];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int p = 32 * t + 8 * (k >> 2) + 4 * h + (k & 3);
            const int64_t row = min(p, c.s - 1);
            float(&mm)[V] = m[t][k >> 3][k >> 2 & 1][k & 3];
            float(&gg)[V] = g[t][k >> 3][k >> 2 & 1][k & 3];
            if constexpr (TAIL) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int x = min(x0 + V * j + v, end - 1);
                    mm[v] = *as_global(at.mom + row * at.mom_pitch + x);
                    gg[v] = load_grad<BF16>(at.grad, row * at.grad_pitch + x);
                }
            } else {
                load_floats<V>(at.mom + row * at.mom_pitch + x0 + V * j, mm);
                load_grads<BF16, V>(at.grad, row * at.grad_pitch + x0 + V * j, gg);
            }
        }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int p = 32 * t + 8 * (k >> 2) + 4 * h + (k & 3);
                const float n = nesterov_input<BF16>(m[t][k >> 3][k >> 2 & 1][k & 3][v], g[t][k >> 3][k >> 2 & 1][k & 3][v],
                                                     c, factor);
                const bool in = p < c.s && (!TAIL || x0 + V * j + v < end);
                o.n[v][t][k >> 3][k >> 2 & 1][k & 3] = in ? n : 0.0f;
            }
}
// Tall: row x0 + j of memory; vec: runs of 4 T elements lie inside or outside as a whole.
template <int T, bool BF16>
__device__ __forceinline__ void load_tall(Column<T, 1> &o, const Place &at, const BlockCall &c, float factor, int x0,
                                          int end, int j, int h, bool vec) {
    const int64_t row = min(x0 + j, end - 1);
    const float *m0 = at.mom + row * at.mom_pitch;
    const int64_t g0 = row * at.grad_pitch;
    float m[4][4 * T], g[4][4 * T];
    if (vec) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int first = T * (8 * k + 4 * h);
            const int p = first < c.s ? first : 0;
            load_floats<4 * T>(m0 + p, m[k]);
            load_grads<BF16, 4 * T>(at.grad, g0 + p, g[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < 4 * T; ++e) {
                const int p = min(T * (8 * k + 4 * h) + e, c.s - 1);
                m[k][e] = *as_global(m0 + p);
                g[k][e] = load_grad<BF16>(at.grad, g0 + p);
            }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const bool in = T * (8 * k + 4 * h + b) + t < c.s && x0 + j < end;
                const float n = nesterov_input<BF16>(m[k][T * b + t], g[k][T * b + t], c, factor);
                o.n[0][t][k >> 1][k & 1][b] = in ? n : 0.0f;
            }
}

// P's fragments in shared memory.
template <int T> struct Poly {
    half8 hi[T][2 * T][64], lo[T][2 * T][64];
    __device__ __forceinline__ void load(const _Float16 *src) {
        const half8 *from = reinterpret_cast<const half8 *>(src);
        half8 *to = &hi[0][0][0];
        for (int k = threadIdx.x; k < T * T * 256; k += kThreads) to[k] = from[k];
    }
};

// The fragment of chunk (t, q) of a column, scaled by a power of two.
template <int T, int V>
__device__ __forceinline__ void column_fragment(const Column<T, V> &o, int v, int t, int q, int shift, half8 &hi, half8 &lo) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = ldexpf(o.n[v][t][q][e >> 2][e & 3], shift);
    split_half(x, hi, lo);
}

// (P N)^T: 32 columns of N as rows, T tiles of 32 basis indices.
template <int T>
__device__ __forceinline__ void times_poly(floatx16 (&acc)[T], const Column<T, 1> &n, const Poly<T> &poly, int lane, int shift) {
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[t][r] = 0.0f;
#pragma unroll
    for (int c = 0; c < 2 * T; ++c) {
        half8 hi, lo;
        column_fragment(n, 0, c >> 1, c & 1, shift, hi, lo);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const half8 bh = poly.hi[t][c][lane], bl = poly.lo[t][c][lane];
            acc[t] = mfma(hi, bh, acc[t]);
            acc[t] = mfma(lo, bh, acc[t]);
            acc[t] = mfma(hi, bl, acc[t]);
        }
    }
}

// One part of one block: the sum of X X^T, X = P N / ||N||, over the part's columns.
template <int T, bool TALL, bool BF16>
__global__ __launch_bounds__(kThreads) void blocks_regram_kernel(const BlockTable t, const BlockCall c) {
    union Shared {
        Poly<T> poly;
        float sums[2 * kWaves * 1024];
    };
    __shared__ __attribute__((aligned(16))) Shared sh;
    const uint32_t block = blockIdx.x / c.parts, part = blockIdx.x % c.parts;  // block: of the launch
    const Place at = locate<BF16 ? 2 : 4, 2>(t, c, c.base + block);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, j = lane & 31, h = lane >> 5;
    const int begin = part * c.part_len, end = min(begin + c.part_len, c.l);
    const float factor = c.factor ? *c.factor : 1.0f;
    const BlockScalars k = c.w.scalars[block];
    const float scale = c.poly_scale * k.inv_norm * kScaleX;
    const bool vec = c.s % (4 * T) == 0;
    sh.poly.load(c.w.poly + static_cast<int64_t>(block) * (T * T * 2048));
    __syncthreads();
    Triangle<T> sum;
    sum.clear();
    for (int x0 = begin + 32 * wave; x0 < end; x0 += kBlockUnit) {
        Column<T, 1> n;
        if constexpr (TALL)
            load_tall<T, BF16>(n, at, c, factor, x0, end, j, h, vec);
        else if (x0 + 32 <= end)
            load_wide<T, 1, BF16, false>(n, at, c, factor, x0, end, j, h);
        else
            load_wide<T, 1, BF16, true>(n, at, c, factor, x0, end, j, h);
        floatx16 acc[T];
        times_poly<T>(acc, n, sh.poly, lane, k.shift);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            half8 hi[T], lo[T];
#pragma unroll
            for (int i = 0; i < T; ++i) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = acc[i][8 * q + e] * scale;
                split_half(x, hi[i], lo[i]);
            }
            sum.add(hi, lo);
        }
    }
    __syncthreads();
    sum.reduce(c.w.gram + (static_cast<int64_t>(block) * c.parts + part) * tri(T) * 1024, sh.sums);
}

// W <- fl(fl(d W) - fl(s O)), O also to ns_out.  N elements that lie side by side.
template <bool PBF16, int N>
__device__ __forceinline__ void update_run(const Place &at, int64_t row, int col, const float (&o)[N], float d, float s) {
    if constexpr (PBF16) {
        uint16_t *p = reinterpret_cast<uint16_t *>(at.param) + row * at.param_pitch + col;
        if constexpr (N == 1 || N == 3) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float w = bf16_bits_to_float(as_global(p)[k]);
                as_global(p)[k] = float_to_bf16_bits(d * w - s * o[k]);
            }
        } else {
            typedef typename HalvesAt<N>::type __attribute__((address_space(1))) *place;
            auto v = *(place)p;
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = float_to_bf16_bits(d * bf16_bits_to_float(v[k]) - s * o[k]);
            *(place)p = v;
        }
    } else {
        float *p = reinterpret_cast<float *>(at.param) + row * at.param_pitch + col;
        float w[N];
        load_floats<N>(p, w);
#pragma unroll
        for (int k = 0; k < N; ++k) w[k] = d * w[k] - s * o[k];
        store_floats<N>(p, w);
    }
    if (at.out) store_floats<N>(at.out + row * at.out_pitch + col, o);
}

template <int T, bool TALL, bool BF16, bool PBF16>
__global__ __launch_bounds__(kThreads) void blocks_update_kernel(const BlockTable t, const BlockCall c) {
    __shared__ __attribute__((aligned(16))) Poly<T> poly;
    const uint32_t block = blockIdx.x / c.parts, part = blockIdx.x % c.parts;  // block: of the launch
    const Place at = locate<BF16 ? 2 : 4, PBF16 ? 2 : 4>(t, c, c.base + block);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, j = lane & 31, h = lane >> 5;
    const int begin = part * c.part_len, end = min(begin + c.part_len, c.l);
    const float factor = c.factor ? *c.factor : 1.0f;
    const BlockScalars k = c.w.scalars[block];
    const float scale = c.poly_scale * k.inv_norm;
    poly.load(c.w.poly + static_cast<int64_t>(block) * (T * T * 2048));
    __syncthreads();
    if constexpr (TALL) {
        const bool vec = c.s % (4 * T) == 0, vec_out = c.s % T == 0;
        for (int x0 = begin + 32 * wave; x0 < end; x0 += kBlockUnit) {
            Column<T, 1> n;
            load_tall<T, BF16>(n, at, c, factor, x0, end, j, h, vec);
            floatx16 acc[T];
            times_poly<T>(acc, n, poly, lane, k.shift);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int x = x0 + acc_row(r, h);
                if (x >= end || T * j >= c.s) continue;
                float o[T];
#pragma unroll
                for (int i = 0; i < T; ++i) o[i] = acc[i][r] * scale;
                if (vec_out || T * j + T <= c.s) {
                    update_run<PBF16, T>(at, x, T * j, o, c.decay, k.update);
                } else {
#pragma unroll
                    for (int i = 0; i < T; ++i) {
                        const float one[1] = {o[i]};
                        if (T * j + i < c.s) update_run<PBF16, 1>(at, x, T * j + i, one, c.decay, k.update);
                    }
                }
            }
        }
    } else {
        // two columns a lane: 4-byte accesses of bf16 gradients and weights
        constexpr int V = 2;
        for (int x0 = begin + 32 * V * wave; x0 < end; x0 += V * kBlockUnit) {
            const bool full = x0 + 32 * V <= end;
            Column<T, V> n;
            if (full)
                load_wide<T, V, BF16, false>(n, at, c, factor, x0, end, j, h);
            else
                load_wide<T, V, BF16, true>(n, at, c, factor, x0, end, j, h);
            floatx16 acc[V][T];
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < T; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[v][i][r] = 0.0f;
#pragma unroll
            for (int q = 0; q < 2 * T; ++q) {
                half8 hi[V], lo[V];
#pragma unroll
                for (int v = 0; v < V; ++v) column_fragment(n, v, q >> 1, q & 1, k.shift, hi[v], lo[v]);
#pragma unroll
                for (int i = 0; i < T; ++i) {
                    const half8 ah = poly.hi[i][q][lane], al = poly.lo[i][q][lane];
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[v][i] = mfma(ah, hi[v], acc[v][i]);
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[v][i] = mfma(ah, lo[v], acc[v][i]);
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[v][i] = mfma(al, hi[v], acc[v][i]);
                }
            }
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int p = 32 * i + acc_row(r, h), x = x0 + V * j;
                    if (p >= c.s) continue;
                    float o[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) o[v] = acc[v][i][r] * scale;
                    if (full) {
                        update_run<PBF16, V>(at, p, x, o, c.decay, k.update);
                    } else {
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            const float one[1] = {o[v]};
                            if (x + v < end) update_run<PBF16, 1>(at, p, x + v, one, c.decay, k.update);
                        }
                    }
                }
        }
    }
}

// Calls fn with the kernel's T, TALL and gradient type as constants.
template <class F> hipError_t choose(int tiles, bool tall, bool bf16, F fn) {
    auto types = [&](auto t) -> hipError_t {
        if (tall) return bf16 ? fn(t, std::true_type{}, std::true_type{}) : fn(t, std::true_type{}, std::false_type{});
        return bf16 ? fn(t, std::false_type{}, std::true_type{}) : fn(t, std::false_type{}, std::false_type{});
    };
    switch (tiles) {
        case 1: return types(std::integral_constant<int, 1>{});
        case 2: return types(std::integral_constant<int, 2>{});
        case 3: return types(std::integral_constant<int, 3>{});
        case 4: return types(std::integral_constant<int, 4>{});
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_blocks_momentum(const BlockTable &t, const BlockCall &c, uint32_t blocks, bool tall, bool grad_bf16,
                                  hipStream_t st) {
    return choose(block_tiles(c.s), tall, grad_bf16, [&](auto tiles, auto is_tall, auto bf16) {
        hipLaunchKernelGGL((blocks_momentum_kernel<tiles.value, is_tall.value, bf16.value>), dim3(blocks * c.parts),
                           dim3(kThreads), 0, st, t, c);
        return hipGetLastError();
    });
}

hipError_t launch_blocks_regram(const BlockTable &t, const BlockCall &c, uint32_t blocks, bool tall, bool grad_bf16,
                                hipStream_t st) {
    return choose(block_tiles(c.s), tall, grad_bf16, [&](auto tiles, auto is_tall, auto bf16) {
        hipLaunchKernelGGL((blocks_regram_kernel<tiles.value, is_tall.value, bf16.value>), dim3(blocks * c.parts),
                           dim3(kThreads), 0, st, t, c);
        return hipGetLastError();
    });
}

hipError_t launch_blocks_update(const BlockTable &t, const BlockCall &c, uint32_t blocks, bool tall, bool grad_bf16,
                                bool param_bf16, hipStream_t st) {
    return choose(block_tiles(c.s), tall, grad_bf16, [&](auto tiles, auto is_tall, auto bf16) {
        if (param_bf16)
            hipLaunchKernelGGL((blocks_update_kernel<tiles.value, is_tall.value, bf16.value, true>),
                               dim3(blocks * c.parts), dim3(kThreads), 0, st, t, c);
        else
            hipLaunchKernelGGL((blocks_update_kernel<tiles.value, is_tall.value, bf16.value, false>),
                               dim3(blocks * c.parts), dim3(kThreads), 0, st, t, c);
        return hipGetLastError();
    });
}

hipError_t launch_blocks_chain(const BlockChain &c, uint32_t blocks, hipStream_t st) {
    switch (block_tiles(c.s)) {
        case 1: hipLaunchKernelGGL(blocks_chain_kernel<1>, dim3(blocks), dim3(64), 0, st, c); break;
        case 2: hipLaunchKernelGGL(blocks_chain_kernel<2>, dim3(blocks), dim3(128), 0, st, c); break;
        case 3: hipLaunchKernelGGL(blocks_chain_kernel<3>, dim3(blocks), dim3(192), 0, st, c); break;
        case 4: hipLaunchKernelGGL(blocks_chain_kernel<4>, dim3(blocks), dim3(256), 0, st, c); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace muon
