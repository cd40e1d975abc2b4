// hc_pre_bwd.h -- gradients of hc_mixes_pre: sizes shared by its kernels and
// the ABI's workspace rule.
#pragma once

#include "hc_kept.cuh"

namespace hc {

// Per-token coefficients that the first kernel leaves for the second, in
// floats: pre [HC], q, padding to HC + 4; comb [HC][HC]; du [(2+HC) HC].
template <int HC>
struct Coef {
    static constexpr int kMix = (2 + HC) * HC;
    static constexpr int kQ = HC, kComb = HC + 4, kDu = HC + 4 + HC * HC;
    static constexpr int kFloats = kDu + kMix;
    static_assert(kFloats % 4 == 0, "rows of whole 16-byte pieces");
};

struct PreBackward {
    int64_t n, d;
    int hc, iters;
    float eps, norm_eps;
    const uint16_t *dy;                    // [n, d]
    Kept x;                                // [n, hc, d]
    const float *mixes, *w, *scale, *base;
    const float *dpost, *dcomb;
    const uint16_t *dstream;               // [n, hc, d] or null
    uint16_t *dx;                          // [n, hc, d]; may be dstream
    float *dw, *dscale, *dbase;
    uint8_t *ws;                           // pre_backward_bytes
};

constexpr int kBackwardMaxIters = 256;  // Sinkhorn divisors kept in shared memory

size_t pre_backward_bytes(int64_t n, int hc, int64_t d);
cudaError_t launch_pre_backward(const PreBackward &p, const DeviceInfo &di, cudaStream_t s);

}  // namespace hc
