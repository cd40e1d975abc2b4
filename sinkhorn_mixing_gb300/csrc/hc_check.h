// hc_check.h -- host-side argument checks shared by the ABI's source files.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <initializer_list>

#include "../../include/hcmix.h"

namespace hc {
namespace check {

inline bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
    uintptr_t lo, hi;
};
inline Range rng(const void *p, uint64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + (uintptr_t)bytes};
}
inline bool overlap(const Range &a, const Range &b) {
    return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo;
}

inline bool finite_nonneg(float v) { return v >= 0.0f && v < INFINITY; }

// Shape checks shared by the entry points that take d.
inline hc_status check_shape(int64_t n, int hc, int64_t d) {
    if (n < 0 || d <= 0) return HC_ERR_INVALID_ARG;
    if (hc != 4 && hc != 8) return HC_ERR_UNSUPPORTED;
    if (d % 8 != 0) return HC_ERR_MISALIGNED;
    // keep every byte count well inside int64: n <= 2^40, d <= 2^24
    if (n > (int64_t(1) << 40) || d > (int64_t(1) << 24)) return HC_ERR_UNSUPPORTED;
    return HC_OK;
}

inline hc_status check_hc_n(int64_t n, int hc) {
    if (n < 0) return HC_ERR_INVALID_ARG;
    if (hc != 4 && hc != 8) return HC_ERR_UNSUPPORTED;
    if (n > (int64_t(1) << 40)) return HC_ERR_UNSUPPORTED;
    return HC_OK;
}

inline hc_status ptrs_ok(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (p == nullptr) return HC_ERR_INVALID_ARG;
    for (const void *p : ps)
        if (!al16(p)) return HC_ERR_MISALIGNED;
    return HC_OK;
}

// Every output range must be disjoint from every other listed range.
inline bool disjoint(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (auto a = outs.begin(); a != outs.end(); ++a) {
        for (auto b = a + 1; b != outs.end(); ++b)
            if (overlap(*a, *b)) return false;
        for (const Range &b : ins)
            if (overlap(*a, b)) return false;
    }
    return true;
}

// A CUDA call or launch has failed.  The runtime keeps its error until someone asks for it, and
// the next call's launch does (launched()): it is taken away here, with the call it belongs to.
inline hc_status cuda_failed() {
    (void)cudaGetLastError();
    return HC_ERR_CUDA;
}
inline hc_status from_cuda(cudaError_t e) { return e == cudaSuccess ? HC_OK : cuda_failed(); }

}  // namespace check
}  // namespace hc
