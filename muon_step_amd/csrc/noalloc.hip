// Fixed device scratch of the allocation-free variant of muon_step, for
// callers that cannot allocate device memory during a step (code under HIP
// graph capture, tight serving loops, harnesses that forbid allocation).
//
// One static array per GPU the library runs on, held until the process ends.
// In host code the name `scratch` is only a host-side stand-in: the device
// address of each GPU's copy comes from hipGetSymbolAddress, called once per
// device by muon_create with that device current, and only that address is
// ever handed to kernels or copies.
//
// Under capture the call's descriptors travel as kernel arguments instead of
// through the context's staging memory: a copy node would read that memory at
// every replay, when a later call may have filled it with other matrices.
#include <algorithm>

#include "kernels.hpp"

static __device__ __align__(256) char scratch[muon::kScratchBytes];

namespace muon {

namespace {

// Descriptors of one launch, passed by value: below 4 KB of arguments.
constexpr int kDescs = 80;
struct Descs {
    MatDesc d[kDescs];
};
static_assert(sizeof(Descs) + 64 <= 4096, "kernel arguments");

__global__ __launch_bounds__(kDescs) void write_descs_kernel(MatDesc *dst, const Descs t, int n) {
    if (static_cast<int>(threadIdx.x) < n) dst[threadIdx.x] = t.d[threadIdx.x];
}

}  // namespace

hipError_t launch_write_descs(MatDesc *dst, const MatDesc *src, int64_t count, hipStream_t st) {
    for (int64_t i = 0; i < count; i += kDescs) {
        const int n = static_cast<int>(std::min<int64_t>(kDescs, count - i));
        Descs t{};
        std::copy(src + i, src + i + n, t.d);
        hipLaunchKernelGGL(write_descs_kernel, dim3(1), dim3(kDescs), 0, st, dst + i, t, n);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

hipError_t scratch_address(void **out) { return hipGetSymbolAddress(out, HIP_SYMBOL(scratch)); }

}  // namespace muon
