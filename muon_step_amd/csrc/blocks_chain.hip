// The polynomials of the block step (blocks.hpp).
#include "blocks_device.hpp"

namespace muon {

namespace {

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
    half8 ah[2][T], al[2][T];
    auto fetch = [&](int c) {
#pragma unroll
        for (int i = 0; i < T; ++i) {
            ah[c & 1][i] = left.hi[i][c][lane];
            al[c & 1][i] = left.lo[i][c][lane];
        }
    };
    fetch(0);
#pragma unroll
    for (int c = 0; c < 2 * T; ++c) {
        if (c + 1 < 2 * T) fetch(c + 1);
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = b.v[c >> 1][8 * (c & 1) + e] * scale;
        half8 hi, lo;
        split_half(x, hi, lo);
#pragma unroll
        for (int i = 0; i < T; ++i) acc[i] = mfma(ah[c & 1][i], hi, acc[i]);
#pragma unroll
        for (int i = 0; i < T; ++i) acc[i] = mfma(ah[c & 1][i], lo, acc[i]);
#pragma unroll
        for (int i = 0; i < T; ++i) acc[i] = mfma(al[c & 1][i], hi, acc[i]);
        __builtin_amdgcn_sched_barrier(0);
    }
    Slab<T> r;
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k) r.v[i][k] = acc[i][k] * out;
    return r;
}

template <int T> __global__ __launch_bounds__(64 * T, 1) void blocks_chain_kernel(const BlockChain c) {
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

    // P: the identity, or what the segments before made it.  Its rows and columns
    // past the smaller side stay zero, whatever N is taken to be there.
    const bool there = c.tall ? T * j + wave < c.s : col < c.s;
    Slab<T> p;
    float *own = c.w.poly_own + (block * T + wave) * T * 1024;
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            p.v[t][r] = c.first ? (on_diagonal(t, r) && there ? 1.0f : 0.0f) : own[(t * 16 + r) * 64 + lane];

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

}  // namespace

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
