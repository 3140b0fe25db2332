// The block step's first two passes for blocks with a smaller side of at most 16, such
// as the factors of an adapter: sums and polynomials in fp64.
//
// A block of this side is a single tile of v_mfma_f64_16x16x4, and the whole schedule
// needs no Gram matrix but the first: fp64's rounding, 2^-53 times a^2 a step, stays
// small where the longest schedule ends (a gain of 2^22, squared: 2^-9 of a vanishing
// direction). What is left of the error is P's and N's rounding in the last product:
// 1.5e-6 of O on spectra over three decades, as an fp32 iteration in X has (1e-6), where
// fp16 pairs in two segments leave 1.3e-5; on even spectra 1.5e-7.
//
// Bound by latency: 27 blocks of 16 x 2048, fp32, take 6.0 us for the sums and 11.7 for
// ten steps, 16 matrix instructions each that wait for one another four at a time; with
// the last pass 21.8 us a call, where two segments of fp16 pairs took 41.2. 1600 blocks
// of 16 x 256 take 56 us (90), 600 of 16 x 4096 266 (354).
//
// Fragments.  Either operand of v_mfma_f64_16x16x4 is, in lane (i, h), i < 16, h < 4,
// entry k = h of row (column) i; the result holds in register r of lane (j, h) row
// 4 r + h of column j.  So a result's register r is the right operand of chunk r as it
// is, and as the left one that of the transpose: L^T R takes four instructions and
// nothing leaves its lane, which is what the congruences of blocks_chain.hip ask for.
#include "blocks_device.hpp"

namespace muon {

namespace {

typedef double double4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ double4_t mfma64(double a, double b, double4_t c) {
    return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

// ---------------------------------------------------------------- momentum

// M and G of 32 columns of X.  Lane (i, h) holds eight entries of basis index i: in
// wide blocks columns 8 h .. 8 h + 7, side by side in memory, in tall ones rows 8 h ..
// 8 h + 7.  Lanes past the smaller side read its last entry.
template <bool TALL, bool BF16> struct Strip {
    static constexpr bool kPacked = BF16 && !TALL;
    float m[8];
    uint32_t g[kPacked ? 4 : 8];

    __device__ __forceinline__ void load(const Place &at, int i, int x) {
        if constexpr (TALL) {
#pragma unroll
            for (int e = 0; e < 8; ++e) one(at, i, x, e);
        } else {
            const float *from = at.mom + i * at.mom_pitch + x;
#pragma unroll
            for (int k = 0; k < 8; k += 4) {
                const auto v = *(const typename WordsAt<4, 4>::type __attribute__((address_space(1))) *)(from + k);
#pragma unroll
                for (int q = 0; q < 4; ++q) m[k + q] = __uint_as_float(v[q]);
            }
            const char *grad = at.grad + (i * at.grad_pitch + x) * (BF16 ? 2 : 4);
#pragma unroll
            for (int k = 0; k < (BF16 ? 4 : 8); k += 4) {
                const auto v = *(const typename WordsAt<4, BF16 ? 2 : 4>::type __attribute__((address_space(1))) *)(grad + 4 * k);
#pragma unroll
                for (int q = 0; q < 4; ++q) g[k + q] = v[q];
            }
        }
    }
    // The same of columns that may end within the strip: others are read as the last one.
    __device__ __forceinline__ void load_part(const Place &at, int i, int x, int end) {
#pragma unroll
        for (int e = 0; e < 8; ++e) one(at, i, min(x + e, end - 1) - e, e);
    }
    __device__ __forceinline__ float grad(int e) const {
        if constexpr (kPacked) return __uint_as_float(e % 2 ? g[e / 2] & 0xffff0000u : g[e / 2] << 16);
        return __uint_as_float(BF16 ? g[e] << 16 : g[e]);
    }

  private:
    __device__ __forceinline__ void one(const Place &at, int i, int x, int e) {
        const int64_t row = TALL ? x + e : i, col = TALL ? i : x + e;
        m[e] = as_global(at.mom)[row * at.mom_pitch + col];
        const int64_t from = row * at.grad_pitch + col;
        if constexpr (BF16) {
            const uint32_t v = as_global(reinterpret_cast<const uint16_t *>(at.grad))[from];
            if constexpr (kPacked)
                g[e / 2] = e % 2 ? g[e / 2] | v << 16 : v;
            else
                g[e] = v;
        } else {
            g[e] = as_global(reinterpret_cast<const uint32_t *>(at.grad))[from];
        }
    }
};

// One part of one block: M <- mu M + G and the sum of N N^T over the part's columns.
template <bool TALL, bool BF16>
__global__ __launch_bounds__(kThreads) void narrow_momentum_kernel(const BlockTable t, const BlockCall c) {
    __shared__ double sh[kWaves][256];
    const uint32_t block = blockIdx.x / c.parts, part = blockIdx.x % c.parts;  // block: of the launch
    const Place at = locate<BF16 ? 2 : 4, 2>(t, c, c.base + block);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, h = lane >> 4;
    const bool mine = (lane & 15) < c.s;
    const int i = min(lane & 15, c.s - 1);
    const int begin = part * c.part_len, end = min(begin + c.part_len, c.l);
    const float factor = c.factor ? *c.factor : 1.0f, mu = c.mu;
    const bool nesterov = c.nesterov != 0;
    double4_t sum = {0.0, 0.0, 0.0, 0.0};
    // `there` of the lane's eight columns are in the part
    auto add = [&](Strip<TALL, BF16> &in, int x, int there) {
        double n[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float g = in.grad(e) * factor;
            float &v = in.m[e];
            v = mu * v + g;
            n[e] = mine && e < there ? static_cast<double>(nesterov ? __builtin_fmaf(mu, v, g) : v) : 0.0;
        }
        if (mine) {
            float *to = at.mom + (TALL ? x * at.mom_pitch + i : i * at.mom_pitch + x);
            if (!TALL && there >= 8) {
#pragma unroll
                for (int k = 0; k < 8; k += 4) {
                    const typename WordsAt<4, 4>::type v = {__float_as_uint(in.m[k]), __float_as_uint(in.m[k + 1]),
                                                            __float_as_uint(in.m[k + 2]), __float_as_uint(in.m[k + 3])};
                    *(typename WordsAt<4, 4>::type __attribute__((address_space(1))) *)(to + k) = v;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < there) as_global(to)[e * (TALL ? at.mom_pitch : 1)] = in.m[e];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = mfma64(n[e], n[e], sum);
    };
    const int whole = begin + (end - begin) / 32 * 32;
    int x0 = begin + 32 * wave;
    Strip<TALL, BF16> next;
    if (x0 < whole) next.load(at, i, x0 + 8 * h);
    for (; x0 < whole; x0 += kBlockUnit) {
        Strip<TALL, BF16> in = next;
        if (x0 + kBlockUnit < whole) next.load(at, i, x0 + kBlockUnit + 8 * h);
        add(in, x0 + 8 * h, 8);
    }
    if (x0 < end) {  // the strip that the part ends in
        next.load_part(at, i, x0 + 8 * h, end);
        add(next, x0 + 8 * h, end - x0 - 8 * h);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) sh[wave][64 * r + lane] = sum[r];
    __syncthreads();
    double all = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) all += sh[w][threadIdx.x];
    as_global(c.w.narrow)[(static_cast<int64_t>(block) * c.parts + part) * 256 + threadIdx.x] = all;
}

// ---------------------------------------------------------------- polynomials

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off, 64);
    return x;
}
// L^T R.
__device__ __forceinline__ double4_t product(const double4_t &left, const double4_t &right) {
    double4_t out = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int r = 0; r < 4; ++r) out = mfma64(left[r], right[r], out);
    return out;
}

// All steps of one block, and P's rows as the last pass reads them.
__global__ __launch_bounds__(64) void narrow_chain_kernel(const NarrowChain c) {
    __shared__ __attribute__((aligned(16))) float rows[32][36];
    const int lane = threadIdx.x, j = lane & 15, h = lane >> 4;
    const int64_t block = blockIdx.x;
    double4_t a = {0.0, 0.0, 0.0, 0.0}, p, unit;
    const double *from = c.w.narrow + block * c.parts * 256 + lane;
#pragma unroll 4
    for (int k = 0; k < c.parts; ++k)
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r] += as_global(from)[256 * k + 64 * r];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        unit[r] = 4 * r + h == j ? 1.0 : 0.0;
        p[r] = j < c.s ? unit[r] : 0.0;  // rows and columns past the smaller side stay zero
    }
    double trace = 0.0;
#pragma unroll
    for (int r = 0; r < 4; ++r) trace += unit[r] != 0.0 ? a[r] : 0.0;
    trace = wave_sum(trace);  // squares of fp32 values neither vanish nor overflow
    const bool zero = trace == 0.0, bad = !(trace < __builtin_inf());
    const double inv = 1.0 / trace;
#pragma unroll
    for (int r = 0; r < 4; ++r) a[r] *= inv;
    double square = 1.0;  // ||O||^2
    for (int k = 0; k < c.steps; ++k) {
        const NarrowChain::Step step = c.step[k];
        const double4_t s = product(a, a);
        double4_t q;
#pragma unroll
        for (int r = 0; r < 4; ++r) q[r] = step.a * unit[r] + step.b * a[r] + step.c * s[r];
        const double4_t ar = product(a, q);
        p = product(q, p);
        if (k + 1 == c.steps) {  // ||O||^2 = tr Q A Q
            square = 0.0;
#pragma unroll
            for (int r = 0; r < 4; ++r) square += q[r] * ar[r];
            square = wave_sum(square);
        }
        a = product(q, ar);
    }
    // P's fragments as P 2^-poly: its largest entry below 2^15, and P N below 2^15
    float most = 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) most = fmaxf(most, fabsf(static_cast<float>(p[r])));
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor(most, off, 64));
    const int poly = max(__builtin_amdgcn_frexp_expf(most) - 15, c.poly_least);
    if (lane == 0) {
        const double norm = sqrt(trace);
        const int e = zero || bad ? 0 : ilogb(sqrt(static_cast<double>(c.s) * c.l) / norm);
        const double o = sqrt(square);
        BlockScalars out;
        out.shift = e;
        out.inv_norm = zero || bad ? 1.0f : static_cast<float>(1.0 / ldexp(norm, e));
        out.update = !c.unit_rms ? c.update : zero || !(o > 0.0) ? 0.0f : static_cast<float>(c.update / o);
        out.poly = poly;
        c.w.scalars[block] = out;
    }
    for (int k = lane; k < 32 * 36; k += 64) (&rows[0][0])[k] = 0.0f;
    __syncthreads();
    const float nan = __builtin_nanf("");
#pragma unroll
    for (int r = 0; r < 4; ++r)
        rows[4 * r + h][j] = zero ? 0.0f : bad ? nan : static_cast<float>(ldexp(p[r], -poly));
    __syncthreads();
    store_poly<1>(c.w.poly, block, rows, 0, lane);
}

}  // namespace

hipError_t launch_narrow_momentum(const BlockTable &t, const BlockCall &c, uint32_t blocks, bool tall, bool grad_bf16,
                                  hipStream_t st) {
    const dim3 grid(blocks * c.parts), threads(kThreads);
    if (tall) {
        if (grad_bf16)
            hipLaunchKernelGGL((narrow_momentum_kernel<true, true>), grid, threads, 0, st, t, c);
        else
            hipLaunchKernelGGL((narrow_momentum_kernel<true, false>), grid, threads, 0, st, t, c);
    } else {
        if (grad_bf16)
            hipLaunchKernelGGL((narrow_momentum_kernel<false, true>), grid, threads, 0, st, t, c);
        else
            hipLaunchKernelGGL((narrow_momentum_kernel<false, false>), grid, threads, 0, st, t, c);
    }
    return hipGetLastError();
}

hipError_t launch_narrow_chain(const NarrowChain &c, uint32_t blocks, hipStream_t st) {
    hipLaunchKernelGGL(narrow_chain_kernel, dim3(blocks), dim3(64), 0, st, c);
    return hipGetLastError();
}

}  // namespace muon
