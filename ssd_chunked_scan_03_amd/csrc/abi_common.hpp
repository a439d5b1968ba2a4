// abi_common.hpp -- what the C ABI units share: shape checks, alignment and overlap tests,
// and the kernels of empty problems.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "device.hpp"
#include "ssd.h"

namespace {

using ssd::grid_ok;
using ssd::kMaxThreads;

// hT = h0 (or 0) for an empty sequence: a fill kernel, not a memset, so that the
// call stays safe under stream capture.
__global__ void k_copy_state(const float* __restrict__ h0, float* __restrict__ hT, int64_t n) {
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) hT[i] = h0 ? h0[i] : 0.f;
}
// (The states may hold more elements than the 2^32 - 1 threads of a launch, past which a launch
// covers their remainder and reports nothing.)
int copy_state(const float* src, float* dst, int64_t n, void* stream) {
    const int64_t blocks = (n + 255) / 256, most = 1 << 20;
    k_copy_state<<<(unsigned)(blocks < most ? blocks : most), 256, 0, (hipStream_t)stream>>>(src, dst, n);
    return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP;
}

// dst[0 .. n) = 0: the empty-problem values of the backward's parameter gradients
__global__ void k_zero(float* __restrict__ dst, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) dst[i] = 0.f;
}

constexpr size_t kAlign = 256;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

bool pn_supported(int64_t P, int64_t N) {
    const bool p = P == 16 || P == 32 || P == 64 || P == 128;
    const bool n = N == 16 || N == 32 || N == 64 || N == 128 || N == 256;
    return p && n;
}

size_t esize(int32_t dtype) { return dtype == SSD_BF16 ? 2 : 4; }

// Shape checks shared by every entry point.
int check_problem(const ssd_problem* p) {
    if (!p) return SSD_ERR_NULL;
    if (p->batch < 0 || p->seqlen < 0 || p->nheads <= 0 || p->headdim <= 0 || p->dstate <= 0 ||
        p->ngroups <= 0 || p->chunk <= 0)
        return SSD_ERR_SHAPE;
    if (p->nheads % p->ngroups != 0) return SSD_ERR_SHAPE;
    if (p->dtype != SSD_F32 && p->dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (p->chunk != 64 && p->chunk != 128 && p->chunk != 256) return SSD_ERR_UNSUPPORTED;
    if (!pn_supported(p->headdim, p->dstate)) return SSD_ERR_UNSUPPORTED;
    if (p->flags & ~(SSD_STAGE_ALL | SSD_SCHEDULE_SPLIT | SSD_SCHEDULE_FUSED)) return SSD_ERR_UNSUPPORTED;
    if ((p->flags & SSD_SCHEDULE_SPLIT) && (p->flags & SSD_SCHEDULE_FUSED)) return SSD_ERR_UNSUPPORTED;
    // launch-grid limits: blocks per launch and the batch / group grid dimensions
    const int64_t nc = (p->seqlen + p->chunk - 1) / p->chunk;
    if (p->batch > 65535 || p->batch * p->ngroups > 65535) return SSD_ERR_UNSUPPORTED;
    // the preparation launches' second grid dimension: ceil(nheads / 16) cumsum tasks plus
    // at most 28 table tasks per group (the backward's, at chunk 256)
    if ((p->nheads + 15) / 16 + 28 * p->ngroups > 65535) return SSD_ERR_UNSUPPORTED;
    if (p->nheads > (int64_t)1 << 20 || nc > (int64_t)1 << 24) return SSD_ERR_UNSUPPORTED;
    if (p->batch * p->nheads * (nc > 0 ? nc : 1) > 0x7fffffffLL) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

bool aligned(const void* ptr, size_t a) { return ((uintptr_t)ptr % a) == 0; }

struct Range {
    const void* p;
    size_t n;
};
bool overlap(Range a, Range b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

}  // namespace
