// The polynomials of the block step (blocks.hpp), for sides above 16.
//
// One workgroup for each block, T waves with 32 columns of every matrix each, which
// stay in registers; the common left operand goes through shared memory.  Bound by
// latency: a step is three products, each of which waits for the other waves'
// columns (two barriers; the matrix cores are busy for 36% of the time), and by the
// matrix cores only when blocks outnumber the CUs.  Both chains of the hybrid schedule
// take 128 us for 16 blocks of 128, 123 for 128 of them, 950 for 1728; 1% of it goes into
// P's scales.
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
// One wave's columns as operand fragments.
template <int T> struct Pairs {
    half8 hi[2 * T], lo[2 * T];
};
template <int T> __device__ __forceinline__ void split_chunk(const Slab<T> &m, int c, half8 &hi, half8 &lo) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = m.v[c >> 1][8 * (c & 1) + e];
    split_half<true>(x, hi, lo);
}
// left^T times the columns whose fragments `right(b, c, hi, lo)` gives, for B
// right operands at once; every chunk's fragments are fetched and split during
// the chunk before it.
template <int T, int B, class F>
__device__ __forceinline__ void product(floatx16 (&acc)[B][T], const Left<T> &left, int lane, F right) {
    half8 ah[2][T], al[2][T], bh[2][B], bl[2][B];
    auto fetch = [&](int c) {
#pragma unroll
        for (int i = 0; i < T; ++i) {
            ah[c & 1][i] = left.hi[i][c][lane];
            al[c & 1][i] = left.lo[i][c][lane];
        }
#pragma unroll
        for (int b = 0; b < B; ++b) right(b, c, bh[c & 1][b], bl[c & 1][b]);
    };
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[b][i][r] = 0.0f;
    fetch(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < 2 * T; ++c) {
        if (c + 1 < 2 * T) fetch(c + 1);
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int b = 0; b < B; ++b)
#pragma unroll
                for (int i = 0; i < T; ++i)
                    acc[b][i] = mfma(k == 2 ? al[c & 1][i] : ah[c & 1][i], k == 1 ? bl[c & 1][b] : bh[c & 1][b], acc[b][i]);
        // loads first, then the splits' instructions between those of the matrix core
        __builtin_amdgcn_sched_group_barrier(0x100, 2 * T + 2 * B, 0);
#pragma unroll
        for (int k = 0; k < 3 * B * T; ++k) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <int T> __global__ __launch_bounds__(64 * T, 1) void blocks_chain_kernel(const BlockChain c) {
    union Shared {
        Left<T> left;
        float rows[32 * T][32 * T + 4];
    };
    __shared__ __attribute__((aligned(16))) Shared sh;
    __shared__ float sh_sum[T];
    __shared__ int sh_exp[T];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, j = lane & 31, h = lane >> 5;
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
    auto add_parts = [&](int first, auto count) {
        constexpr int N = count.value;
        floatx4 v[N][T][4];
        float weight[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float *g = c.w.gram + (block * c.parts + first + n) * tri(T) * 1024 + 4 * lane;
#pragma unroll
            for (int t = 0; t < T; ++t)
                if (t >= wave) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        v[n][t][q] = *(const floatx4 __attribute__((address_space(1))) *)(g + (tri(t) + wave) * 1024 + 256 * q);
                }
            weight[n] = 1.0f;
            if (c.first) weight[n] = parts[first + n].largest == 0 ? 0.0f : ldexpf(1.0f, 2 * (parts[first + n].shift - common));
        }
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int t = 0; t < T; ++t)
                if (t >= wave) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) a.v[t][r] = __builtin_fmaf(weight[n], v[n][t][r >> 2][r & 3], a.v[t][r]);
                }
    };
    // some parts' loads at once
    int k = 0;
    for (; k + 4 <= c.parts; k += 4) add_parts(k, std::integral_constant<int, 4>{});
    for (; k < c.parts; ++k) add_parts(k, std::integral_constant<int, 1>{});
    // the tiles above the diagonal, from the waves that hold their mirror images
#pragma unroll
    for (int t = 0; t < T; ++t)
        if (t > wave) {
#pragma unroll
            for (int r = 0; r < 16; ++r) sh.rows[32 * t + acc_row(r, h)][col] = a.v[t][r];
        }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < T; ++t)
        if (t < wave) {
#pragma unroll
            for (int r = 0; r < 16; ++r) a.v[t][r] = sh.rows[col][32 * t + acc_row(r, h)];
        }
    __syncthreads();
    if (c.first) {
        float trace = 0.0f;
#pragma unroll
        for (int t = 0; t < T; ++t)
            if (t == wave) {
#pragma unroll
                for (int r = 0; r < 16; ++r) trace += acc_row(r, h) == j ? a.v[t][r] : 0.0f;
            }
        trace = total(trace);
        const float n = sqrtf(trace), inv = 1.0f / trace;
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) a.v[t][r] *= inv;
        if (threadIdx.x == 0) {
            int e = 0;  // 2^e <= sqrt(s l) / norm < 2^(e + 1)
            (void)frexpf(sqrtf(static_cast<float>(c.s) * static_cast<float>(c.l)) / n, &e);
            --e;
            BlockScalars out;
            out.shift = zero || bad ? 0 : e - common;
            out.inv_norm = zero || bad ? 1.0f : 1.0f / ldexpf(n, e);
            out.update = c.update;
            out.poly = 0;
            c.w.scalars[block] = out;
        }
    } else {
        // the sums are of P's fragments times N 2^shift
        const float scale = __builtin_amdgcn_ldexpf(c.w.scalars[block].inv_norm, c.w.scalars[block].poly);
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) a.v[t][r] = a.v[t][r] * scale * scale;
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
            p.v[t][r] = c.first ? (on_diagonal(t, r) && there ? 1.0f : 0.0f) : as_global(own)[(t * 16 + r) * 64 + lane];

    // P as it enters the products: each column p 2^p_exp, its largest entry p below 2^12
    // and at least half of that.  How large P's entries become goes by the spectrum (by
    // its smallest singular value, up to the schedule's gain, where N has one): a scale
    // for the worst of them would leave an even one's P below fp16's smallest values.
    // A column stays in its lanes as a right operand, so its scale needs no other wave.
    int p_exp = 0;
    auto normalize = [&]() {
        float most = 0.0f;
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) most = fmaxf(most, fabsf(p.v[t][r]));
        most = fmaxf(most, __shfl_xor(most, 32, 64));
        const int up = 12 - __builtin_amdgcn_frexp_expf(most);
        p_exp -= up;
        return __builtin_amdgcn_ldexpf(1.0f, up);
    };
    auto scale_p = [&](float by) {
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) p.v[t][r] *= by;
    };
    scale_p(normalize());
    // A and Q as they enter the products: A 64, Q 16, A Q 1024.
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) a.v[t][r] *= kScaleA;
    float square = 1.0f;  // ||O||^2
    for (int k = 0; k < c.steps; ++k) {
        const BlockChain::Step step = c.step[k];
        const bool more = k + 1 < c.steps, norm = !more && c.last && c.unit_rms;
#pragma unroll
        for (int i = 0; i < 2 * T; ++i) {
            half8 hi, lo;
            split_chunk(a, i, hi, lo);
            sh.left.hi[wave][i][lane] = hi;
            sh.left.lo[wave][i][lane] = lo;
        }
        __syncthreads();
        floatx16 s[1][T];
        // A^T A: the wave's own columns of A are among the rows of A^T
        product<T, 1>(s, sh.left, lane, [&](int, int i, half8 &hi, half8 &lo) {
            hi = sh.left.hi[wave][i][lane];
            lo = sh.left.lo[wave][i][lane];
        });
        const float qa = kScaleQ * step.a, qb = kScaleQ / kScaleA * step.b, qc = kScaleQ / (kScaleA * kScaleA) * step.c;
        Slab<T> q;
#pragma unroll
        for (int t = 0; t < T; ++t) {
#pragma unroll
            for (int r = 0; r < 16; ++r) q.v[t][r] = __builtin_fmaf(qc, s[0][t][r], qb * a.v[t][r]);
            if (t == wave) {
#pragma unroll
                for (int r = 0; r < 16; ++r) q.v[t][r] += acc_row(r, h) == j ? qa : 0.0f;
            }
        }
        Pairs<T> pairs;
        Slab<T> ar;  // A^T Q
        if (more || norm) {
            floatx16 acc[1][T];
            product<T, 1>(acc, sh.left, lane, [&](int, int i, half8 &hi, half8 &lo) {
                split_chunk(q, i, hi, lo);
                pairs.hi[i] = hi;
                pairs.lo[i] = lo;
            });
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) ar.v[t][r] = acc[0][t][r];
        } else {
#pragma unroll
            for (int i = 0; i < 2 * T; ++i) split_chunk(q, i, pairs.hi[i], pairs.lo[i]);
        }
        if (norm) {  // ||O||^2 = tr Q A Q
            float sq = 0.0f;
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) sq += q.v[t][r] * ar.v[t][r];
            square = total(sq) / (kScaleA * kScaleQ * kScaleQ);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2 * T; ++i) {
            sh.left.hi[wave][i][lane] = pairs.hi[i];
            sh.left.lo[wave][i][lane] = pairs.lo[i];
        }
        __syncthreads();
        if (more) {
            floatx16 acc[2][T];
            product<T, 2>(acc, sh.left, lane, [&](int b, int i, half8 &hi, half8 &lo) { split_chunk(b ? ar : p, i, hi, lo); });
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    p.v[t][r] = acc[0][t][r];
                    a.v[t][r] = acc[1][t][r] * (1.0f / (kScaleQ * kScaleQ));
                }
        } else {
            floatx16 acc[1][T];
            product<T, 1>(acc, sh.left, lane, [&](int, int i, half8 &hi, half8 &lo) { split_chunk(p, i, hi, lo); });
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) p.v[t][r] = acc[0][t][r];
        }
        p_exp -= kLogScaleQ;
        scale_p(normalize());
        __syncthreads();
    }

    if (c.last && c.unit_rms && threadIdx.x == 0) {
        const double o = sqrt(static_cast<double>(square));
        c.w.scalars[block].update = zero || !(o > 0) ? 0.0f : static_cast<float>(c.update / o);
    }

    // P's columns for the next segment, and its rows as fragments for the products with
    // N, of P 2^-poly: its largest entry below 2^15, and P N below 2^15.
    int largest_exp = there ? p_exp : -1000;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) largest_exp = max(largest_exp, __shfl_xor(largest_exp, off, 64));
    if (lane == 0) sh_exp[wave] = largest_exp;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < T; ++w) largest_exp = max(largest_exp, sh_exp[w]);
    const int poly = max(largest_exp + 12 - 15, c.poly_least);
    if (threadIdx.x == 0) c.w.scalars[block].poly = poly;
    const float nan = __builtin_nanf("");
    const float whole = __builtin_amdgcn_ldexpf(1.0f, p_exp), part = __builtin_amdgcn_ldexpf(1.0f, p_exp - poly);
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float x = zero ? 0.0f : bad ? nan : p.v[t][r];
            if (!c.last) as_global(own)[(t * 16 + r) * 64 + lane] = x * whole;
            sh.rows[32 * t + acc_row(r, h)][col] = x * part;
        }
    __syncthreads();
    store_poly<T>(c.w.poly, block, sh.rows, wave, lane);
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
