// The balance loss of MoE routers, the tokens that each expert got, the gradient of the
// logits, and the step of the selection biases.
//
// For a sequence s of n tokens (those that take part) whose choices name expert i
// C_i times, p_t a token's normalised scores (softmax, or sigmoids over their sum):
//     loss_s = coef sum_i f_i P_i,   f_i = E C_i / (K n),   P_i = (1 / n) sum_t p_ti
// and the loss is the mean over the sequences that have tokens, S of them.  With
// c_i = coef E C_i / (S K n^2) it is the sum over tokens of sum_i c_i p_ti, and
//     d loss / d x_ti = p_ti (c_i - sum_j c_j p_tj)      times 1 - sigma(x_ti) for sigmoids.
// Counts depend on the choices alone, so one pass over the logits gives loss and
// gradient: count, balance, finish.  As sum_i p_ti = 1, a constant may be taken off
// c_i: off its mean the differences that make up the gradient do not cancel when
// loads are nearly even, and the mean itself goes into the loss.
#include <type_traits>

#include "router.hpp"
#include "tensor_table.hpp"
#include "vector_access.hpp"

namespace muon {

namespace {

constexpr int kWaves = kRouterThreads / 64;

// A sequence's tokens; what offsets leave out of the tokens is left out here.
struct Span {
    int begin, end;
};
__device__ __forceinline__ Span span_of(const RouterDesc &d, int s) {
    if (!d.offsets) return Span{0, d.tokens};
    const int lo = as_global(d.offsets)[s], hi = as_global(d.offsets)[s + 1];
    return Span{max(lo, 0), min(hi, d.tokens)};
}
// The last sequence of [lo, hi] that begins at or before the token.
__device__ __forceinline__ int sequence_of(const RouterDesc &d, int token, int lo, int hi) {
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (as_global(d.offsets)[mid] <= token)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}
// The same for a token that the wave has in common: 64 places are looked at in turn.
__device__ __forceinline__ int wave_sequence_of(const RouterDesc &d, int token) {
    int lo = 0, n = d.offsets ? d.sequences : 1;
    while (n > 1) {
        const int width = (n + 63) / 64, at = lo + static_cast<int>(threadIdx.x & 63) * width;
        const bool begun = at < lo + n && as_global(d.offsets)[at] <= token;
        // the count is unsigned: where no place has begun, one less would be the largest of all
        const int k = max(static_cast<int>(__popcll(__ballot(begun))) - 1, 0);
        n = min(width, n - k * width);
        lo += k * width;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}
__device__ __forceinline__ bool takes_part(const RouterDesc &d, int token, int s) {
    const Span p = span_of(d, s);
    return token >= p.begin && token < p.end && (!d.mask || as_global(d.mask)[token] != 0);
}

// Adds the choices of tokens [begin, end), a token for each thread at a time, to
// `own`, which holds the counts of the sequences from s0 on (`window` of them),
// and to hist past those.  Returns how many sequences the thread has given their first
// token in hist.
__device__ __forceinline__ int count_tokens(const RouterDesc &d, int begin, int end, int s0, int s1, uint32_t *own, int window) {
    const int stride = d.experts + 1, top = d.top_k;
    int found = 0;
    for (int token = begin + threadIdx.x; token < end; token += blockDim.x) {
        const int s = sequence_of(d, token, s0, s1);
        const bool in = takes_part(d, token, s);
        const int64_t at = static_cast<int64_t>(token) * top;
        const bool near = s - s0 < window;
        uint32_t *to = near ? own + (s - s0) * stride : d.hist + static_cast<int64_t>(s) * stride;
        auto add = [&](int i) {
            if (near)
                __hip_atomic_fetch_add((uint32_t __attribute__((address_space(3))) *)(own + (s - s0) * stride + i), 1u,
                                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            else
                atomicAdd(to + i, 1u);
        };
        if (in) {
            if (near)
                add(d.experts);
            else
                found += atomicAdd(to + d.experts, 1u) == 0;
        }
        for (int j0 = 0; j0 < top; j0 += 4) {
            int64_t x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t k = at + min(j0 + j, top - 1);
                x[j] = d.chosen64 ? as_global(static_cast<const int64_t *>(d.chosen))[k]
                                  : as_global(static_cast<const int32_t *>(d.chosen))[k];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (in && j0 + j < top && x[j] >= 0 && x[j] < d.experts) add(static_cast<int>(x[j]));
        }
    }
    return found;
}

// Counts of the sequences that the workgroup's tokens begin with are gathered in
// shared memory, as many as fit there.  Whoever gives a sequence its first token counts
// it as one that has any: the pass over the logits needs their number.  Looking through
// all sequences there, in every workgroup, is no faster where they are few (one layer in 5
// sequences 17.4 us, 17.2 so) and was, with one workgroup to a router in the last launch,
// most of 427 us at 4096 sequences of 256 experts, which take 80 now.
__global__ __launch_bounds__(kRouterThreads) void router_count_kernel(const RouterTable t, const RouterCall c) {
    __shared__ uint32_t own[kCountWords];
    const Owners<64> owners(t.first);
    const int e = owners.of(blockIdx.x);
    const RouterDesc &d = t.d[e];
    const int begin = (blockIdx.x - t.first[e]) * c.per_block, end = min(begin + static_cast<int>(c.per_block), d.tokens);
    if (begin >= end) return;
    const int stride = d.experts + 1;
    const int s0 = wave_sequence_of(d, begin), s1 = wave_sequence_of(d, end - 1);
    const int window = min(kCountWords / stride, s1 - s0 + 1);
    for (int k = threadIdx.x; k < window * stride; k += kRouterThreads) own[k] = 0;
    __syncthreads();
    int found = count_tokens(d, begin, end, s0, s1, own, window);
    __syncthreads();
    uint32_t *hist = d.hist + static_cast<int64_t>(s0) * stride;
    for (int k = threadIdx.x * stride + d.experts; k < window * stride; k += kRouterThreads * stride)
        if (own[k] != 0) {
            found += atomicAdd(hist + k, own[k]) == 0;
            own[k] = 0;
        }
    __syncthreads();
    for (int k = threadIdx.x; k < window * stride; k += kRouterThreads)
        if (own[k] != 0) atomicAdd(hist + k, own[k]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) found += __shfl_xor(found, off, 64);
    if ((threadIdx.x & 63) == 0 && found != 0) atomicAdd(c.live + e, static_cast<uint32_t>(found));
}

// The value of lane ^ OFF, for values that are the same in each OFF neighbours
// already: within 16 lanes by a lane permutation in the instruction itself
// (mirrors serve for 4 and 8), beyond by swaps of halves.
template <int OFF> __device__ __forceinline__ float across(float x) {
    const int v = __float_as_int(x);
    if constexpr (OFF == 1) return __int_as_float(__builtin_amdgcn_mov_dpp(v, 0xb1, 0xf, 0xf, true));   // quad 1 0 3 2
    if constexpr (OFF == 2) return __int_as_float(__builtin_amdgcn_mov_dpp(v, 0x4e, 0xf, 0xf, true));   // quad 2 3 0 1
    if constexpr (OFF == 4) return __int_as_float(__builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true));  // mirror of 8
    if constexpr (OFF == 8) return __int_as_float(__builtin_amdgcn_mov_dpp(v, 0x140, 0xf, 0xf, true));  // mirror of 16
    return __shfl_xor(x, OFF, 64);
}
// Sum and maximum over the LANES lanes of a row, in all of them.
template <int LANES, int OFF = 1> __device__ __forceinline__ float row_sum(float x) {
    if constexpr (OFF < LANES) return row_sum<LANES, 2 * OFF>(x + across<OFF>(x));
    return x;
}
template <int LANES, int OFF = 1> __device__ __forceinline__ float row_max(float x) {
    if constexpr (OFF < LANES) return row_max<LANES, 2 * OFF>(fmaxf(x, across<OFF>(x)));
    return x;
}
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

// A lane of LANES to a row takes PER of its elements, eight side by side and the
// next eight 8 LANES further on: element k is expert 8 lane + at(k).
template <int LANES> __device__ __forceinline__ constexpr int at(int k) { return k / 8 * 8 * LANES + k % 8; }

// The lane's logits of a row as they lie in memory, and as numbers; those past the
// row's end (`there` of them and more, from the lane's first one on) are -inf: their
// score is zero.
template <int LANES, int PER, bool BF16> struct Row {
    static constexpr int kEight = BF16 ? 4 : 8;  // words of eight
    uint32_t w[PER / 8 * kEight];

    __device__ __forceinline__ void load(const void *p, int64_t first, int there) {
        const char *from = static_cast<const char *>(p) + first * (BF16 ? 2 : 4);
#pragma unroll
        for (int s = 0; s < PER / 8; ++s) {
            const char *place = from + at<LANES>(8 * s) * (BF16 ? 2 : 4);
            const int left = there - at<LANES>(8 * s);
            if (left >= 8) {
#pragma unroll
                for (int k = 0; k < kEight; k += 4) {
                    const auto v = *(const typename Words<4, BF16 ? 2 : 4>::type __attribute__((address_space(1))) *)(place + 4 * k);
#pragma unroll
                    for (int q = 0; q < 4; ++q) w[s * kEight + k + q] = v[q];
                }
            } else {
                constexpr uint32_t kNone = BF16 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
                for (int k = 0; k < kEight; ++k) w[s * kEight + k] = kNone;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < left) {
                        if constexpr (BF16) {
                            uint32_t &to = w[s * kEight + k / 2];
                            const uint32_t v = as_global(reinterpret_cast<const uint16_t *>(place))[k];
                            to = k % 2 ? (to & 0xffffu) | v << 16 : (to & 0xffff0000u) | v;
                        } else {
                            w[s * kEight + k] = as_global(reinterpret_cast<const uint32_t *>(place))[k];
                        }
                    }
            }
        }
    }
    __device__ __forceinline__ float operator[](int k) const {
        if constexpr (BF16) return __uint_as_float(k % 2 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
        return __uint_as_float(w[k]);
    }
};
template <int LANES, int PER, bool BF16>
__device__ __forceinline__ void store_row(void *p, int64_t first, int there, const float (&x)[PER]) {
    char *to = static_cast<char *>(p) + first * (BF16 ? 2 : 4);
#pragma unroll
    for (int s = 0; s < PER / 8; ++s) {
        char *place = to + at<LANES>(8 * s) * (BF16 ? 2 : 4);
        const int left = there - at<LANES>(8 * s);
        const float *y = x + 8 * s;
        if (left >= 8) {
            if constexpr (BF16) {
                const uint32_t w[4] = {pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                       pack_bf16x2(y[6], y[7])};
                store_words<4, 2>(place, w);
            } else {
#pragma unroll
                for (int k = 0; k < 8; k += 4) {
                    const uint32_t w[4] = {__float_as_uint(y[k]), __float_as_uint(y[k + 1]), __float_as_uint(y[k + 2]),
                                           __float_as_uint(y[k + 3])};
                    store_words<4, 4>(place + 4 * k, w);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < left) {
                    if constexpr (BF16)
                        as_global(reinterpret_cast<uint16_t *>(place))[k] = float_to_bf16_bits(y[k]);
                    else
                        as_global(reinterpret_cast<float *>(place))[k] = y[k];
                }
        }
    }
}

// What a lane needs of its row's sequence: its span, and how far the factors of the
// lane's experts lie from their mean.
template <int PER> struct Factors {
    int s = -1;
    Span span{0, 0};
    float away[PER], mean = 0.0f;
};

// Gradients of tokens [begin, end), LANES lanes to a row of up to LANES x PER
// logits, 64 / LANES rows a wave, and the lane's part of the loss.  hist: counts of
// the sequences from s0 on; `live`: how many sequences have tokens.
template <int LANES, int PER, bool BF16, bool SIGMOID>
__device__ __forceinline__ double balance_rows(const RouterDesc &d, const RouterCall &c, const uint32_t *hist, int begin, int end,
                                               int s0, int s1, int live) {
    constexpr int kRows = 64 / LANES;
    const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int row0 = lane / LANES, i0 = lane % LANES * 8;  // the lane's row of a wave's rows, and its first expert
    const int stride = d.experts + 1, there = d.experts - i0;
    const float grad_scale = c.grad_scale ? *as_global(c.grad_scale) : 1.0f;
    double loss = 0.0;
    Factors<PER> f;
#pragma unroll
    for (int k = 0; k < PER; ++k) f.away[k] = 0.0f;

    auto find = [&](int token) {
        f.s = sequence_of(d, token, max(f.s, s0), s1);
        f.span = span_of(d, f.s);
        const uint32_t *h = hist + static_cast<int64_t>(f.s - s0) * stride;
        const double n = h[d.experts];
        double total = 0.0;
        uint32_t got[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            got[k] = at<LANES>(k) < there ? h[i0 + at<LANES>(k)] : 0;
            total += got[k];
        }
#pragma unroll
        for (int off = 1; off < LANES; off *= 2) total += __shfl_xor(total, off, 64);
        const double unit = n > 0 ? c.coef / (static_cast<double>(live) * d.top_k * n * n) : 0.0;
        f.mean = static_cast<float>(unit * total);
#pragma unroll
        for (int k = 0; k < PER; ++k)
            f.away[k] = at<LANES>(k) < there ? static_cast<float>(unit * (static_cast<double>(d.experts) * got[k] - total)) : 0.0f;
    };
    // a wave's next rows are on their way while it works on these
    Row<LANES, PER, BF16> next;
    uint8_t next_mask = 1;
    auto fetch = [&](int base) {
        const int token = min(base + row0, end - 1);
        next.load(d.logits, static_cast<int64_t>(token) * d.pitch + i0, there);
        next_mask = d.mask ? as_global(d.mask)[token] : 1;
    };
    int base = begin + wave * kRows;
    if (base < end) fetch(base);
    for (; base < end; base += waves * kRows) {
        const int token = base + row0;
        Row<LANES, PER, BF16> x = next;
        const bool unmasked = next_mask != 0;
        if (base + waves * kRows < end) fetch(base + waves * kRows);
        if (token < end && (f.s < 0 || token >= f.span.end)) find(token);
        const bool inside = token < end && token >= f.span.begin && token < f.span.end;
        const bool taking = inside && unmasked;
        // w: a score, not yet normalised; q: its derivative's factor
        float w[PER], q[PER], sum, dot;
        auto shifted = [&](float (&to)[PER]) {  // exp(x - max)
            float most = -3.402823466e38f;
#pragma unroll
            for (int k = 0; k < PER; ++k) most = fmaxf(most, x[k]);
            most = row_max<LANES>(most);
#pragma unroll
            for (int k = 0; k < PER; ++k) to[k] = exp_of(x[k] - most);
        };
        auto add = [&]() {
            sum = 0.0f;
            dot = 0.0f;
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                sum += w[k];
                dot = __builtin_fmaf(f.away[k], w[k], dot);
            }
            sum = row_sum<LANES>(sum);
            dot = row_sum<LANES>(dot);
        };
        if constexpr (SIGMOID) {
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                // sigma and 1 - sigma, each without cancellation.  v_rcp_f32 gives zero for what lies below the
                // smallest normal number: a sigma below 1.18e-38 is zero, as one of a logit of -infinity is
                const float e = exp_of(-x[k]);
                w[k] = __builtin_amdgcn_rcpf(1.0f + e);
                q[k] = fminf(e, 3e38f) * w[k];  // a NaN is one in w
            }
            if (there < at<LANES>(PER - 1) + 1) {
#pragma unroll
                for (int k = 0; k < PER; ++k) w[k] = at<LANES>(k) < there ? w[k] : 0.0f;
            }
            add();
            // rows whose sigmoids are all small: there sigma(x) is exp(x) and 1 - sigma(x) is 1, to fp32's last bit,
            // and no score need be below the smallest normal number
            const bool vanish = taking && sum < 0x1p-26f;
            if (__any(vanish)) {
                float other[PER];
                shifted(other);
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    w[k] = vanish ? other[k] : w[k];
                    q[k] = vanish ? 1.0f : q[k];
                }
                add();
            }
        } else {
            shifted(w);
            add();
        }
        // a row without any score: no probability, no gradient
        const float inv = sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sum);
        dot *= inv;
        if (taking && lane % LANES == 0) loss += static_cast<double>(dot) + (sum == 0.0f ? 0.0f : f.mean);
        if (inside && d.dlogits) {
            float g[PER];
            const float scale = inv * grad_scale, off = -dot * scale;
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                g[k] = w[k] * __builtin_fmaf(f.away[k], scale, off);
                if constexpr (SIGMOID) g[k] *= q[k];
            }
            if (!taking) {
#pragma unroll
                for (int k = 0; k < PER; ++k) g[k] = 0.0f;
            }
            store_row<LANES, PER, BF16>(d.dlogits, static_cast<int64_t>(token) * d.dpitch + i0, there, g);
        }
    }
    return loss;
}

// Sum over the workgroup, in thread 0.
__device__ __forceinline__ double block_sum(double x, double *sh) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x += __shfl_down(x, off, 64);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
    __syncthreads();
    double sum = 0.0;
    if (threadIdx.x == 0)
        for (uint32_t k = 0; k < blockDim.x >> 6; ++k) sum += sh[k];
    return sum;
}
template <int LANES, int PER, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(kRouterThreads) void router_balance_kernel(const RouterTable t, const RouterCall c) {
    __shared__ double sh_sum[kWaves];
    const Owners<64> owners(t.first);
    const int e = owners.of(blockIdx.x);
    const RouterDesc &d = t.d[e];
    const uint32_t mine = blockIdx.x - t.first[e];
    if (mine == 0 && !c.accumulate)  // what the next launch adds to
        for (int i = threadIdx.x; i < d.experts; i += kRouterThreads) as_global(d.counts)[i] = 0;
    const int begin = mine * c.per_block, end = min(begin + static_cast<int>(c.per_block), d.tokens);
    const int s0 = wave_sequence_of(d, begin), s1 = wave_sequence_of(d, end - 1);
    const int live = static_cast<int>(as_global(c.live)[e]);
    const double loss = balance_rows<LANES, PER, BF16, SIGMOID>(d, c, d.hist + static_cast<int64_t>(s0) * (d.experts + 1), begin,
                                                                end, s0, s1, live);
    const double sum = block_sum(loss, sh_sum);
    if (threadIdx.x == 0) d.sums[mine] = sum;
}

// How many of the sequences have tokens, by their counts in shared memory.
__device__ __forceinline__ int live_sequences(const RouterDesc &d, const uint32_t *hist, int *sh) {
    if (threadIdx.x == 0) *sh = 0;
    __syncthreads();
    int found = 0;
    for (int s = threadIdx.x; s < d.sequences; s += blockDim.x) found += hist[s * (d.experts + 1) + d.experts] != 0;
    if (found) atomicAdd(sh, found);
    __syncthreads();
    return *sh;
}

// Small batches: one workgroup for each router does all of it, counts in shared memory.
template <int LANES, int PER, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(kSmallThreads) void router_small_kernel(const RouterTable t, const RouterCall c) {
    __shared__ uint32_t hist[kCountWords];
    __shared__ double sh_sum[kSmallThreads / 64];
    __shared__ int sh_live;
    const RouterDesc &d = t.d[blockIdx.x];
    const int stride = d.experts + 1;
    for (int k = threadIdx.x; k < d.sequences * stride; k += kSmallThreads) hist[k] = 0;
    __syncthreads();
    count_tokens(d, 0, d.tokens, 0, d.offsets ? d.sequences - 1 : 0, hist, d.sequences);
    __syncthreads();
    const int live = live_sequences(d, hist, &sh_live);
    const double loss = balance_rows<LANES, PER, BF16, SIGMOID>(d, c, hist, 0, d.tokens, 0, d.offsets ? d.sequences - 1 : 0, live);
    const double sum = block_sum(loss, sh_sum);
    if (threadIdx.x == 0) *d.loss = static_cast<float>(sum);
    for (int i = threadIdx.x; i < d.experts; i += kSmallThreads) {
        int64_t n = 0;
        for (int s = 0; s < d.sequences; ++s) n += hist[s * stride + i];
        as_global(d.counts)[i] = c.accumulate ? as_global(d.counts)[i] + n : n;
    }
}

// One workgroup for each router and `slices` times kFinishWords of its counts, in
// whole sequences: adds them up by experts and leaves them at zero; the first one
// adds up the loss.
__global__ __launch_bounds__(kFinishThreads) void router_finish_kernel(const RouterTable t, uint32_t blocks, uint32_t slices,
                                                                       const RouterCall c) {
    __shared__ double sh_sum[kFinishThreads / 64];
    __shared__ unsigned long long counts[kMaxExperts + 1];
    const int e = blockIdx.x;
    const RouterDesc &d = t.d[e];
    const uint32_t next = e + 1 < kRouters ? min(t.first[e + 1], blocks) : blocks, count = next - t.first[e];
    const uint32_t stride = d.experts + 1;
    const int64_t slice = static_cast<int64_t>(finish_sequences(d.experts)) * slices * stride;
    const int64_t begin = blockIdx.y * slice, end = min(begin + slice, static_cast<int64_t>(d.sequences) * stride);
    if (blockIdx.y > 0 && begin >= end) return;
    for (uint32_t i = threadIdx.x; i < stride; i += kFinishThreads) counts[i] = 0;
    __syncthreads();
    uint32_t i = threadIdx.x % stride;
    const uint32_t turn = kFinishThreads % stride;
    for (int64_t k = begin + threadIdx.x; k < end; k += kFinishThreads) {
        const uint32_t n = as_global(d.hist)[k];
        if (n != 0) {
            atomicAdd(&counts[i], static_cast<unsigned long long>(n));
            as_global(d.hist)[k] = 0;
        }
        i += turn;
        if (i >= stride) i -= stride;
    }
    double sum = 0.0;
    if (blockIdx.y == 0)
        for (uint32_t k = threadIdx.x; k < count; k += kFinishThreads) sum += as_global(d.sums)[k];
    sum = block_sum(sum, sh_sum);  // (a barrier for the counts, too)
    // of several workgroups each adds to the zeros that the pass over the logits has left (if it had any tokens)
    const bool write = (gridDim.y == 1 || count == 0) && !c.accumulate;
    for (uint32_t k = threadIdx.x; k < stride - 1; k += kFinishThreads) {
        if (write)
            as_global(d.counts)[k] = static_cast<int64_t>(counts[k]);
        else if (counts[k] != 0)
            atomicAdd(reinterpret_cast<unsigned long long *>(d.counts) + k, counts[k]);
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) {
        *d.loss = static_cast<float>(sum);
        as_global(c.live)[e] = 0;
    }
}

__global__ __launch_bounds__(kRouterThreads) void router_clear_kernel(uint32_t *p, int64_t words, uint32_t *live) {
    if (blockIdx.x == 0 && threadIdx.x < kRouters) live[threadIdx.x] = 0;
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * kRouterThreads + threadIdx.x; k < words;
         k += static_cast<int64_t>(gridDim.x) * kRouterThreads)
        p[k] = 0;
}

// b_i <- b_i - rate sign(C_i - mean C), the comparison in whole numbers.
__global__ __launch_bounds__(kRouterThreads) void router_bias_kernel(const RouterBiasTable t, float rate) {
    __shared__ int64_t sh_sum[kWaves];
    const RouterBiasDesc &d = t.d[blockIdx.x];
    int64_t total = 0;
    for (int64_t i = threadIdx.x; i < d.experts; i += kRouterThreads) total += as_global(d.counts)[i];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) total += __shfl_xor(total, off, 64);
    if ((threadIdx.x & 63) == 0) sh_sum[threadIdx.x >> 6] = total;
    __syncthreads();
    total = 0;
    for (int k = 0; k < kWaves; ++k) total += sh_sum[k];
    for (int64_t i = threadIdx.x; i < d.experts; i += kRouterThreads) {
        const int64_t excess = d.experts * as_global(d.counts)[i] - total;
        const float step = excess > 0 ? -rate : excess < 0 ? rate : 0.0f;
        as_global(d.bias)[i] += step;
    }
}

template <int LANES, int PER, bool BF16, bool SIGMOID>
hipError_t launch_as(const RouterTable &t, uint32_t blocks, const RouterCall &c, bool small, hipStream_t st) {
    if (small)
        hipLaunchKernelGGL((router_small_kernel<LANES, PER, BF16, SIGMOID>), dim3(blocks), dim3(kSmallThreads), 0, st, t, c);
    else
        hipLaunchKernelGGL((router_balance_kernel<LANES, PER, BF16, SIGMOID>), dim3(blocks), dim3(kRouterThreads), 0, st, t, c);
    return hipGetLastError();
}
template <int LANES, int PER>
hipError_t launch_rows(const RouterTable &t, uint32_t blocks, const RouterCall &c, bool bf16, bool small, hipStream_t st) {
    if (c.sigmoid)
        return bf16 ? launch_as<LANES, PER, true, true>(t, blocks, c, small, st)
                    : launch_as<LANES, PER, false, true>(t, blocks, c, small, st);
    return bf16 ? launch_as<LANES, PER, true, false>(t, blocks, c, small, st)
                : launch_as<LANES, PER, false, false>(t, blocks, c, small, st);
}
hipError_t launch_any(const RouterTable &t, uint32_t blocks, const RouterCall &c, int experts, bool bf16, bool small,
                      hipStream_t st) {
    if (experts <= 32) {
        switch (router_lanes(experts)) {
            case 1: return launch_rows<1, 8>(t, blocks, c, bf16, small, st);
            case 2: return launch_rows<2, 8>(t, blocks, c, bf16, small, st);
            default: return launch_rows<4, 8>(t, blocks, c, bf16, small, st);
        }
    }
    switch (router_lanes(experts)) {
        case 4: return launch_rows<4, 16>(t, blocks, c, bf16, small, st);
        case 8: return launch_rows<8, 16>(t, blocks, c, bf16, small, st);
        case 16: return launch_rows<16, 16>(t, blocks, c, bf16, small, st);
        case 32: return launch_rows<32, 16>(t, blocks, c, bf16, small, st);
        default: return launch_rows<64, 16>(t, blocks, c, bf16, small, st);
    }
}

}  // namespace

hipError_t launch_router_count(const RouterTable &t, uint32_t blocks, const RouterCall &c, hipStream_t st) {
    hipLaunchKernelGGL(router_count_kernel, dim3(blocks), dim3(kRouterThreads), 0, st, t, c);
    return hipGetLastError();
}

hipError_t launch_router_balance(const RouterTable &t, uint32_t blocks, const RouterCall &c, int experts, bool bf16,
                                 hipStream_t st) {
    return launch_any(t, blocks, c, experts, bf16, false, st);
}

hipError_t launch_router_small(const RouterTable &t, int routers, const RouterCall &c, int experts, bool bf16, hipStream_t st) {
    return launch_any(t, routers, c, experts, bf16, true, st);
}

hipError_t launch_router_finish(const RouterTable &t, int routers, uint32_t blocks, const RouterCall &c, hipStream_t st) {
    uint32_t most = 1;
    for (int i = 0; i < routers; ++i) {
        const uint32_t each = finish_sequences(t.d[i].experts), of = (t.d[i].sequences + each - 1) / each;
        most = of > most ? of : most;
    }
    const uint32_t slices = (most + kFinishSlices - 1) / kFinishSlices;
    hipLaunchKernelGGL(router_finish_kernel, dim3(routers, (most + slices - 1) / slices), dim3(kFinishThreads), 0, st, t, blocks,
                       slices, c);
    return hipGetLastError();
}

hipError_t launch_router_clear(uint32_t *p, int64_t words, uint32_t *live, hipStream_t st) {
    const int64_t blocks = (words + kRouterThreads - 1) / kRouterThreads;
    hipLaunchKernelGGL(router_clear_kernel, dim3(static_cast<uint32_t>(blocks < 1024 ? blocks : 1024)), dim3(kRouterThreads), 0,
                       st, p, words, live);
    return hipGetLastError();
}

hipError_t launch_router_bias(const RouterBiasTable &t, int routers, float rate, hipStream_t st) {
    hipLaunchKernelGGL(router_bias_kernel, dim3(routers), dim3(kRouterThreads), 0, st, t, rate);
    return hipGetLastError();
}

}  // namespace muon
